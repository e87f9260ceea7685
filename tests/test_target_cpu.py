"""Host-side checks of the target pass's operators that need no GPU: refused
arguments, workspace sizes, the page lookup and the node walk that the kernels
share, and the rotation table."""
import ctypes
import math

import numpy as np
import pytest
import torch

import target_reference as ref
from speculative_decoding_verification_70_gb300 import _binding as bd
from test_abi_cpu import lib, needs_no_gpu  # noqa: F401

OK, INVALID, DTYPE, WORKSPACE = 0, 1, 2, 6
P = 1 << 20  # made-up device address (16-byte aligned), never reached


def _kv(**kw):
    f = dict(k=P, v=P, k_page=16 * 8 * 128, k_slot=8 * 128, k_head=128, v_page=16 * 8 * 128, v_slot=8 * 128,
             v_head=128, dtype=1, num_pages=10, page_size=16, Hkv=8, D=128, page_table=P, table_stride=4,
             max_pages=4)
    f.update(kw)
    return bd._pack_kv(*(f[k] or 0 for k in f))


def _nodes(**kw):
    f = dict(B=2, N=4, ctx_len=P, parent=None, n_nodes=None)
    f.update(kw)
    return bd._pack_nodes(*(f[k] or 0 for k in f))


BAD_KV = [dict(k=None), dict(v=P + 2), dict(page_table=None), dict(page_table=P + 2), dict(num_pages=0),
          dict(page_size=0), dict(Hkv=0), dict(D=96), dict(D=256), dict(max_pages=0), dict(table_stride=3),
          dict(k_slot=1028), dict(v_page=0), dict(k_head=-128), dict(k_head=64), dict(v_slot=1 << 40),
          dict(page_size=1 << 20, max_pages=1 << 12, table_stride=1 << 12)]
BAD_NODES = [dict(B=0), dict(N=0), dict(N=65), dict(ctx_len=None), dict(parent=P + 1), dict(B=1 << 30)]


def _attend(lib, kv=None, nodes=None, Hq=16, q=P, q_b=4 * 16 * 128, q_n=16 * 128, q_h=128, scale=0.1, out=P,
            lse=P, ws=P, n=1 << 40):
    kv, nodes = kv or _kv(), nodes or _nodes()
    return lib.ssd_tree_attention(kv, nodes, Hq, q, q_b, q_n, q_h, scale, out, lse,
                                  ws, n, None)


def _append(lib, kv=None, nodes=None, Hq=16, q=P, k=P, v=P, q_out=P, cos_sin=P, max_pos=99, rot=128, qn=P, kn=P,
            eps=1e-6, ws=P, n=256, q_b=99, kv_h=128):
    kv, nodes = kv or _kv(), nodes or _nodes()
    return lib.ssd_kv_append(kv, nodes, Hq, q, q_b, 128, 128, k, v, 512, 128, kv_h,
                             q_out, cos_sin, max_pos, rot, 0, qn, kn, eps, ws, n, None)


@needs_no_gpu
@pytest.mark.parametrize("kw", BAD_KV, ids=str)
def test_bad_cache_is_refused(lib, kw):
    assert _attend(lib, kv=_kv(**kw)) == INVALID
    assert _append(lib, kv=_kv(**kw)) == INVALID
    kv = _kv(**kw)
    assert lib.ssd_kv_commit(kv, 1, 0, 0, 2, 4, P, P, P, P + 64, P, 256, None) == INVALID


@needs_no_gpu
@pytest.mark.parametrize("kw", BAD_NODES, ids=str)
def test_bad_nodes_are_refused(lib, kw):
    assert _attend(lib, nodes=_nodes(**kw)) == INVALID
    assert _append(lib, nodes=_nodes(**kw)) == INVALID


@needs_no_gpu
def test_attention_refusals(lib):
    assert _attend(lib, kv=_kv(dtype=0)) == DTYPE
    for kw in (dict(Hq=12), dict(Hq=4), dict(Hq=8 * 65), dict(q=None), dict(q=P + 8), dict(q_n=1028),
               dict(q_b=-8), dict(scale=math.nan), dict(scale=math.inf), dict(out=None), dict(out=P + 8),
               dict(lse=P + 2), dict(ws=None), dict(ws=P + 16)):
        assert _attend(lib, **kw) == INVALID, kw
    need = lib.ssd_tree_attention_workspace_bytes(2, 4, 16, 8, 128)
    assert need >= 256 and _attend(lib, n=need - 1) == WORKSPACE
    assert lib.ssd_tree_attention(None, None, 16, P, 8, 8, 8, 1.0, P, P, P, need, None) == INVALID
    for a in ((0, 1, 1, 1, 64), (1, 65, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 1, 1, 80), (1, 1, 65, 1, 64)):
        assert lib.ssd_tree_attention_workspace_bytes(*a) == 0


@needs_no_gpu
def test_append_refusals(lib):
    assert _append(lib, kv=_kv(dtype=0)) == DTYPE
    for kw in (dict(Hq=0), dict(q=None), dict(q=P + 1), dict(v=P + 1), dict(q_out=P + 8), dict(q_out=None),
               dict(cos_sin=None), dict(rot=0), dict(rot=24), dict(rot=144), dict(max_pos=0), dict(cos_sin=P + 4),
               dict(qn=None), dict(kn=None), dict(eps=-1.0), dict(eps=math.nan), dict(ws=None), dict(q_b=-1),
               dict(kv_h=-1)):
        assert _append(lib, **kw) == INVALID, kw
    assert _append(lib, n=255) == WORKSPACE


@needs_no_gpu
def test_commit_refusals(lib):
    kv = _kv()

    def call(layers=2, kl=1 << 20, vl=1 << 20, B=2, N=4, ctx=P, acc=P, node=P, new=P + 64, ws=P, n=256):
        return lib.ssd_kv_commit(kv, layers, kl, vl, B, N, ctx, acc, node, new, ws, n, None)
    for kw in (dict(layers=0), dict(kl=4), dict(vl=0), dict(B=0), dict(N=65), dict(ctx=None), dict(acc=None),
               dict(new=None), dict(new=P), dict(node=P + 2), dict(ws=None)):
        assert call(**kw) == INVALID, kw
    assert call(n=8) == WORKSPACE


@needs_no_gpu
def test_logprobs_refusals(lib):
    def call(z=P, dt=0, stride=1000, n_rows=5, V=1000, rows=None, R=5, tok=P, T=P, K=4, lp=P, H=P, rk=P, tt=P, tl=P,
             ws=P, n=1 << 40):
        return lib.ssd_logprobs(z, dt, stride, n_rows, V, rows, R, tok, T, K, lp, H, rk, tt, tl, ws, n, None)
    assert call(dt=2) == DTYPE and call(dt=7) == DTYPE
    for kw in (dict(z=None), dict(z=P + 2), dict(stride=999), dict(n_rows=0), dict(V=0), dict(V=1 << 29), dict(R=0),
               dict(R=6), dict(tok=None), dict(tok=P + 2), dict(K=-1), dict(K=33), dict(tt=None), dict(tl=None),
               dict(lp=None), dict(ws=None), dict(ws=P + 4)):
        assert call(**kw) == INVALID, kw
    assert call(n=0) == WORKSPACE
    assert lib.ssd_logprobs_workspace_bytes(0, 10, 1) == 0
    assert lib.ssd_logprobs_workspace_bytes(1, 10, 33) == 0


def test_binding_refuses_cpu_tensors_and_shapes():
    c = ref.case(1, 2, 4, 2, 64, 16, 3, torch.bfloat16, 1)
    with pytest.raises(ValueError):
        bd.ssd_tree_attention(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["ctx_len"])
    with pytest.raises(TypeError):
        bd.ssd_tree_attention(c["q"], c["k_cache"].float(), c["v_cache"].float(), c["page_table"], c["ctx_len"])
    with pytest.raises(ValueError):
        bd.ssd_logprobs(torch.zeros(3, 4), torch.zeros(3, dtype=torch.int32))


def test_page_lookup(lib):
    """Bad pages, slots before and beyond the table: refused before any
    address is made of them."""
    row = np.array([3, -1, 7, 8, 0], dtype=np.int32)
    page, off = ctypes.c_int32(), ctypes.c_int32()

    def look(slot, ps=16, pages=8, width=5):
        ok = lib.ssd_selftest_kv_slot(row.ctypes.data, width, pages, ps, slot, ctypes.byref(page), ctypes.byref(off))
        return (page.value, off.value) if ok else None
    assert look(0) == (3, 0) and look(15) == (3, 15) and look(32) == (7, 0) and look(79) == (0, 15)
    assert look(16) is None          # page -1
    assert look(48) is None          # page 8 of 8
    assert look(80) is None and look(-1) is None and look(1 << 40) is None
    assert look(4, ps=1) == (0, 0) and look(5, ps=1) is None
    assert look(41, ps=40) is None and look(80, ps=40) == (7, 0)


def test_node_walk(lib):
    mask, depth = ctypes.c_uint64(), ctypes.c_int32()

    def walk(par, n, j):
        a = None if par is None else np.array(par, dtype=np.int32)
        ok = lib.ssd_selftest_node(None if a is None else a.ctypes.data, n, j, ctypes.byref(mask),
                                   ctypes.byref(depth))
        return (mask.value, depth.value) if ok else None
    assert walk(None, 64, 63) == ((1 << 64) - 1, 63) and walk(None, 3, 0) == (1, 0)
    assert walk(None, 3, 3) is None and walk(None, 0, 0) is None
    g = torch.Generator().manual_seed(2)
    for N in (1, 2, 21, 64):
        par = ref.random_tree(N, g)
        for j, way in enumerate(ref.ways(par, N)):
            assert walk(par, N, j) == (sum(1 << i for i in way), len(way) - 1)
    broken = [-1, 0, 3, 2, 1, 5, -1]
    assert [walk(broken, 7, j) is not None for j in range(7)] == [True, True, False, False, True, False, False]
    assert walk([0, 0], 2, 1) is None and walk([0, 0], 2, 0) is None


def test_rope_table():
    t = bd.rope_table(200001, 64, 500000.0, device="cpu")
    for pos, i in ((0, 0), (1, 3), (200000, 0), (199999, 31)):
        a = math.fmod(pos * 500000.0 ** (-2 * i / 64), 2 * math.pi)
        # the angle in 64 bits is off by about 2^-52 * 200000, its cosine is rounded once
        assert abs(float(t[pos, i]) - math.cos(a)) <= 2 ** -24 + 1e-10
        assert abs(float(t[pos, 32 + i]) - math.sin(a)) <= 2 ** -24 + 1e-10
    with pytest.raises(ValueError):
        bd.rope_table(10, 64, inv_freq=torch.ones(3), device="cpu")
