"""Bounded waits of the target pass's operators that run out: for bytes that no
copy brings.  The kernels end by themselves and say so, and the workspace is
usable afterwards."""
import math

import pytest
import torch

import target_reference as ref
from test_gpu_target import BF, FP, _check_attention

pytestmark = pytest.mark.gpu
LIMIT_US = 2000


@pytest.fixture
def withheld(gpu_lib):
    """Waits run out while it is entered."""
    class Withheld:
        def __enter__(self):
            gpu_lib.selftest_copy_wait(LIMIT_US, True)

        def __exit__(self, *a):
            torch.cuda.synchronize()
            gpu_lib.selftest_copy_wait()
    yield Withheld()
    gpu_lib.selftest_copy_wait()


@pytest.mark.parametrize("dt", [torch.float32, BF])
@pytest.mark.parametrize("K", [0, 5])
@pytest.mark.parametrize("R,V", [(600, 5000), (3, 128256)])
def test_logprobs_of_rows_that_do_not_arrive(gpu_lib, withheld, dt, K, R, V):
    """Whole rows and rows in parts: NaN and -1 and the error bit, no other; then
    the same call is right."""
    z = torch.randn((R, V), generator=torch.Generator().manual_seed(71)).to(dt).cuda()
    tok = torch.zeros(R, dtype=torch.int32, device="cuda")
    good = gpu_lib.ssd_logprobs(z, tok, K)
    assert gpu_lib.get_device_error(good["ws"]) == 0
    with withheld:
        lost = gpu_lib.ssd_logprobs(z, tok, K, ws=good["ws"])
        torch.cuda.synchronize()
    assert gpu_lib.get_device_error(good["ws"], clear=True) == gpu_lib.DEVERR_TIMEOUT
    for key, value in lost.items():
        if key in ("rank", "top_tok"):
            assert bool((value == -1).all()), key
        elif key != "ws":
            assert bool(torch.isnan(value).all()), key
    again = gpu_lib.ssd_logprobs(z, tok, K, ws=good["ws"])
    assert gpu_lib.get_device_error(good["ws"]) == 0
    for key in good:
        if key != "ws":
            assert torch.equal(again[key], good[key]), key


def test_logprobs_that_need_no_copies(gpu_lib, withheld):
    """Rows that are not 16-byte aligned are read by plain loads."""
    z = torch.randn((4, 999), device="cuda")
    tok = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    with withheld:
        r = gpu_lib.ssd_logprobs(z[:, 1:], tok, 3)
        torch.cuda.synchronize()
    assert gpu_lib.get_device_error(r["ws"]) == 0
    want = torch.log_softmax(z[:, 1:].double(), 1)[:, 7]
    assert float((r["logprob"].double() - want).abs().max()) <= 2.0 ** -18 * math.log(999)


@pytest.mark.parametrize("B,N,Hq,Hkv,D,ctx,dt", [
    (1, 1, 4, 1, 64, 900, BF),                                   # one sequence in parts
    (40, 2, 8, 4, 64, tuple(i * 9 for i in range(40)), FP),      # several a block
    (3, 12, 16, 2, 128, (0, 700, 40), BF),                       # 96 rows: split over the warpgroups
    (1, 64, 8, 1, 128, 1000, BF)])                               # two row blocks
def test_attention_over_tiles_that_do_not_arrive(gpu_lib, withheld, B, N, Hq, Hkv, D, ctx, dt):
    """The call ends with the error bit; then the same call is right."""
    c = ref.case(B, N, Hq, Hkv, D, 16, ctx, dt, 72)
    g = ref.to_gpu(c)
    ws = gpu_lib.new_workspace(gpu_lib.tree_attention_workspace_bytes(B, N, Hq, Hkv, D), "cuda")

    def run():
        r = gpu_lib.ssd_tree_attention(g["q"], g["k_cache"], g["v_cache"], g["page_table"], g["ctx_len"],
                                       parent=g["parent"], ws=ws)
        torch.cuda.synchronize()
        return r
    with withheld:
        run()
    assert gpu_lib.get_device_error(ws, clear=True) == gpu_lib.DEVERR_TIMEOUT
    want = _check_attention(gpu_lib, c)
    again = run()
    assert gpu_lib.get_device_error(ws) == 0
    assert torch.equal(again["out"], want["out"]) and torch.equal(again["lse"], want["lse"])
