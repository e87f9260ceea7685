"""Tree attention over more sequences than a block has threads: several a thread
when the batch's tiles are counted, and more than 2^23 of them.

Tolerances as in tests/test_gpu_target.py.
"""
import pytest
import torch

import target_reference as ref
from test_gpu_target import BF, FP, _check_attention, _same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Hq,Hkv,D,dt", [(513, 2, 1, 64, BF), (1024, 4, 2, 64, FP), (1200, 3, 3, 128, BF)])
def test_sequences_beyond_a_block(gpu_lib, B, Hq, Hkv, D, dt):
    """Two and three sequences a thread; long ones and ones without tiles between
    them, so that ranges begin inside any of a thread's sequences."""
    ctx = [(b * 37) % 41 for b in range(B)]
    for b in range(5, B, 211):
        ctx[b] = 700 + b
    c = ref.case(B, 2, Hq, Hkv, D, 16, ctx, dt, 61, fill="nan")
    n = torch.tensor([2 - (b % 2) for b in range(B)], dtype=torch.int32)
    n[7:B:3] = 0                     # one or two of a thread's sequences are empty
    n[300:320] = 0
    n[B - 2:] = 0
    c["n_nodes"] = n
    r = _check_attention(gpu_lib, c)
    assert gpu_lib.get_device_error(r["ws"]) == 0
    c["n_nodes"] = torch.zeros_like(n)
    c["n_nodes"][B - 3] = 2          # one sequence alone
    _check_attention(gpu_lib, c)


def test_more_than_2_to_the_23_sequences(gpu_lib):
    """Single tokens over up to 14 slots each, pages shared by many."""
    B, D, ps = (1 << 23) + 1000, 64, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(62)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=BF)
    k, v, q = randn(100, ps, 1, D), randn(100, ps, 1, D), randn(B, 1, 1, D)
    table = torch.randint(0, 100, (B, 1), generator=gen, device="cuda").to(torch.int32)
    ctx = torch.randint(0, 15, (B,), generator=gen, device="cuda").to(torch.int32)
    r = gpu_lib.ssd_tree_attention(q, k, v, table, ctx)
    assert gpu_lib.get_device_error(r["ws"]) == 0
    slot = torch.arange(ps, device="cuda")
    half = ref.HALF_STEP[BF]
    for b in range(0, B, 1 << 18):
        at = table[b:b + (1 << 18), 0].long()
        kk, vv, qq = k[at, :, 0].double(), v[at, :, 0].double(), q[b:b + (1 << 18), 0, 0].double()
        s = (kk @ qq[:, :, None])[..., 0] * D ** -0.5
        d = (D + 4) * 2.0 ** -24 * (kk.abs() @ qq.abs()[:, :, None])[..., 0].amax(1) * D ** -0.5
        s = s.masked_fill(slot > ctx[b:b + (1 << 18), None], float("-inf"))
        p = torch.softmax(s, 1)[:, None]
        want, w = (p @ vv)[:, 0], (p @ vv.abs())[:, 0]
        tol = half * want.abs() + w * (half + 2 * d[:, None] + 2.0 ** -18)
        _same(r["out"][b:b + (1 << 18), 0, 0], want.cpu(), tol.cpu(), "out")
        lse = torch.logsumexp(s, 1)
        _same(r["lse"][b:b + (1 << 18), 0, 0], lse.cpu(), (d + 2.0 ** -18 + lse.abs() * 2.0 ** -22).cpu(), "lse")
