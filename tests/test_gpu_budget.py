"""Summed attention weights and eviction against their plain forms in 64 bits."""
import math

import pytest
import torch

import chunk_reference as cref
import target_reference as ref
from test_gpu_chunk import attend, case
from test_gpu_target import _same

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def add_weights(lib, c, lse, w, **kw):
    g = ref.to_gpu(c)
    wg = w.cuda()
    r = lib.ssd_kv_weights(g["q"], g["k_cache"], g["page_table"], g["ctx_len"], lse.cuda(), wg, n_nodes=g["n_nodes"],
                           **kw)
    torch.cuda.synchronize()
    assert r["weights"] is wg
    return r


def check_weights(lib, c, window=0, sinks=0, scale=None, decay=1.0, extra=3, error=0):
    B, H = c["q"].shape[0], c["k_cache"].shape[2]
    S = int(c["ctx_len"].max()) + c["N"] + extra
    w = torch.rand((B, H, S), generator=torch.Generator().manual_seed(1)) * 3
    _, lse, _, _ = cref.attention(c, window, sinks, scale)
    lse = lse.float()
    want, tol = cref.weights(c, lse, w, window, sinks, scale, decay)
    r = add_weights(lib, c, lse, w, window=window, sinks=sinks, scale=scale, decay=decay)
    assert lib.get_device_error(r["ws"]) == error
    _same(r["weights"], want, tol, "weights")
    return r


SUMS = [
    # B, N, Hq, Hkv, D, page, ctx, dtype, ragged, order, window, sinks, decay
    (1, 1, 1, 1, 128, 16, 0, BF, False, "slot", 0, 0, 1.0),
    (2, 1, 8, 2, 128, 16, (127, 128), BF, False, "head", 0, 0, 1.0),
    (2, 1, 64, 1, 64, 16, (127, 128), BF, False, "head", 0, 0, 0.5),
    (3, 8, 8, 2, 128, 16, (120, 121, 500), BF, False, "slot", 100, 4, 0.0),
    (2, 33, 4, 1, 128, 32, (0, 300), FP, True, "head", 0, 0, 0.9),
    (2, 17, 16, 2, 64, 16, (255, 900), BF, False, "slot", 17, 130, 1.0),
    (1, 300, 5, 1, 64, 16, 77, FP, False, "slot", 64, 3, 1.0),
    (2, 140, 14, 2, 128, 64, (0, 129), BF, True, "slot", 0, 0, 0.0),
    (1, 70, 12, 1, 128, 128, 250, BF, False, "head", 0, 0, 1.0),
    (2, 40, 6, 3, 64, 1, (30, 45), BF, False, "slot", 20, 2, 1.0),
    (2, 70, 4, 2, 128, 5, (61, 300), FP, False, "head", 0, 0, -1.0),
    (2, 90, 4, 2, 64, 200, (190, 401), BF, False, "slot", 130, 10, 1.0),
    (1, 30, 4, 2, 128, 256, 300, FP, False, "head", 0, 0, 1.0),
    (70, 2, 4, 2, 64, 16, tuple((i * 37) % 211 for i in range(70)), BF, True, "slot", 0, 0, 1.0),
    (1, 32, 8, 1, 128, 16, 6000, BF, False, "slot", 0, 0, 0.0),
    (3, 500, 2, 2, 128, 48, (0, 1000, 100), FP, True, "slot", 0, 0, 1.0),
    (1, 600, 8, 2, 64, 16, 100, BF, False, "slot", 150, 0, 1.0),
]


@pytest.mark.parametrize("c", SUMS, ids=lambda c: "-".join(str(x) for x in c[:6] + c[10:]))
def test_kv_weights(gpu_lib, c):
    B, N, Hq, Hkv, D, page, ctx, dt, ragged, order, window, sinks, decay = c
    check_weights(gpu_lib, case(B, N, Hq, Hkv, D, page, ctx, dt, 400 + N, ragged, order, width_extra=1), window, sinks,
                  decay=decay)


@pytest.mark.parametrize("scale", [0.3, -0.05, 0.0])
def test_weights_scale_and_packed_queries(gpu_lib, scale):
    for N in (6, 150):
        check_weights(gpu_lib, case(3, N, 8, 2, 128, 16, (5, 90, 200), BF, 7, packed=True), scale=scale)


def test_weights_rows_that_see_nothing(gpu_lib):
    """Rows of lse -inf add nothing; decay 0 does not read what was there."""
    c = case(2, 20, 4, 2, 64, 16, (100, 30), BF, 8)
    _, lse, _, _ = cref.attention(c)
    lse = lse.float()
    lse[0, 3] = -math.inf
    lse[1, :, 2] = -math.inf
    w = torch.full((2, 2, 130), math.nan)
    want, tol = cref.weights(c, lse, w, decay=0.0)
    r = add_weights(gpu_lib, c, lse, w, decay=0.0)
    _same(r["weights"], want, tol, "weights")


def test_weights_lengths_and_pages_out_of_range(gpu_lib):
    lib = gpu_lib
    c = case(5, 6, 4, 2, 128, 16, (20, 33, 50, 7, 9), BF, 11, fill="random")
    c["ctx_len"][0] = -1
    c["n_nodes"] = torch.tensor([6, 7, -1, 6, 6], dtype=torch.int32)
    check_weights(lib, c, error=lib.DEVERR_BAD_LENGTH)
    c = case(2, 6, 4, 2, 128, 16, (40, 100), BF, 12, fill="random")
    check_weights(lib, c, extra=-1, error=lib.DEVERR_BAD_LENGTH)  # one sequence too long for the weights
    c["page_table"][0, 1] = c["k_cache"].shape[0]
    check_weights(lib, c, error=lib.DEVERR_BAD_PAGE)


def test_weights_sum_to_the_rows(gpu_lib):
    """With the attention's own lse every row gives 1 in all."""
    for N, ctx in ((1, 3000), (300, 100)):
        c = case(2, N, 8, 2, 64, 16, ctx, BF, 13)
        r = attend(gpu_lib, c, window=500, sinks=4)
        w = add_weights(gpu_lib, c, r["lse"].cpu(), torch.zeros((2, 2, ctx + N)), window=500, sinks=4, decay=0.0)
        got = w["weights"].double().sum(2).cpu()
        assert float((got / (N * 4) - 1).abs().max()) < 2.0 ** -16


def test_weights_strided_rows_and_same_bits(gpu_lib):
    lib = gpu_lib
    c = ref.to_gpu(case(3, 40, 8, 2, 128, 16, (100, 900, 3), BF, 14))
    lse = lib.ssd_chunk_attention(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["ctx_len"])["lse"]
    big = torch.full((2, 3, 1001), 7.0, device="cuda")
    at = (c["q"], c["k_cache"], c["page_table"], c["ctx_len"], lse)
    w = big.transpose(0, 1)[:, :, 1:]
    lib.ssd_kv_weights(*at, w, decay=0.0)
    flat = torch.full((3, 2, 1000), 7.0, device="cuda")
    ws = lib.ssd_kv_weights(*at, flat, decay=0.0)["ws"]
    assert torch.equal(w, flat) and bool((big[:, :, 0] == 7).all())
    assert bool((flat[0, :, 140:] == 7).all())
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        lib.ssd_kv_weights(*at, flat, decay=0.0, ws=ws)
    for _ in range(3):
        flat.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(w, flat)


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def evict_case(layers, B, Hkv, D, page, ctx, dtype, seed, order="slot", ties=True):
    c = ref.case(B, 1, Hkv, Hkv, D, page, ctx, dtype, seed, tree="chain", order="slot")
    g = torch.Generator().manual_seed(seed)
    shape = (layers,) + (c["k_cache"].shape if order == "slot" else c["k_cache"].transpose(1, 2).shape)
    for n in ("k_cache", "v_cache"):
        t = torch.randn(shape, generator=g).to(dtype)
        c[n] = t if order == "slot" else t.transpose(2, 3)
    S = max(int(c["ctx_len"].max()), 1) + 2
    w = torch.exp(2 * torch.randn((layers, B, Hkv, S), generator=g))
    if ties:
        w = (w * 4).round() / 4
    c["ctx_len"] = torch.tensor(list(ctx) if not isinstance(ctx, int) else [ctx] * B, dtype=torch.int32)
    return c, w


def check_evict(lib, c, w, budget, sinks=0, recent=0, in_place=False, error=0):
    k, v, new, kept, wout = cref.evict(c, w, budget, sinks, recent)
    g = {n: c[n].cuda() if c[n].is_contiguous() else c[n].transpose(2, 3).cuda().transpose(2, 3)
         for n in ("k_cache", "v_cache")}
    wg = w.cuda()
    out = {"weights": wg} if in_place else {"weights": torch.full_like(wg, math.nan)}
    r = lib.ssd_kv_evict(g["k_cache"], g["v_cache"], c["page_table"].cuda(), c["ctx_len"].cuda(), wg, budget,
                         sinks=sinks, recent=recent, out=out)
    torch.cuda.synchronize()
    assert lib.get_device_error(r["ws"]) == error
    assert torch.equal(r["ctx_len"].cpu(), new)
    assert torch.equal(r["kept"].cpu(), kept)
    got = r["weights"].cpu()
    left = torch.isnan(wout).all(3) & ~torch.isnan(w).all(3)  # sequences out of range
    assert torch.equal(got[~left].nan_to_num(-5), wout[~left].nan_to_num(-5))
    assert torch.equal(got[left].nan_to_num(-5), (w if in_place else torch.full_like(w, math.nan))[left].nan_to_num(-5))
    if not in_place:
        assert torch.equal(wg.cpu().nan_to_num(-5), w.nan_to_num(-5))
    assert torch.equal(g["k_cache"].cpu(), k) and torch.equal(g["v_cache"].cpu(), v)


EVICT = [
    # layers, B, Hkv, D, page, ctx, dtype, order, budget, sinks, recent
    (1, 1, 1, 128, 16, 1, BF, "slot", 1, 0, 0),
    (1, 1, 1, 64, 16, 5, BF, "slot", 1, 0, 0),
    (1, 2, 2, 64, 16, (40, 41), BF, "slot", 40, 4, 8),
    (3, 2, 2, 128, 16, (100, 333), BF, "slot", 50, 4, 20),
    (2, 3, 4, 64, 5, (0, 61, 700), FP, "head", 60, 0, 60),
    (2, 3, 4, 64, 1, (10, 61, 700), FP, "head", 60, 60, 0),
    (1, 2, 3, 128, 200, (600, 1300), BF, "slot", 512, 30, 100),
    (1, 2, 8, 128, 64, (4000, 9001), BF, "head", 1000, 16, 64),
    (5, 1, 8, 128, 16, 2049, FP, "slot", 1025, 4, 256),
    (1, 40, 2, 64, 32, tuple((i * 97) % 1100 for i in range(40)), BF, "slot", 300, 4, 100),
    (1, 1, 1, 64, 16, 20011, BF, "slot", 5000, 0, 0),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("c", EVICT, ids=lambda c: "-".join(str(x) for x in c[:6] + c[8:]) if len(str(c[5])) < 30 else "b40")
def test_kv_evict(gpu_lib, c, in_place):
    layers, B, Hkv, D, page, ctx, dt, order, budget, sinks, recent = c
    check_evict(gpu_lib, *evict_case(layers, B, Hkv, D, page, ctx, dt, 500 + budget, order), budget, sinks, recent,
                in_place)


def test_evict_special_weights(gpu_lib):
    """All equal (the lowest stay), zeros of both signs, negative, infinite and NaN ones."""
    c, w = evict_case(1, 2, 2, 64, 16, (300, 777), BF, 20)
    check_evict(gpu_lib, c, torch.ones_like(w), 100, 3, 10)
    check_evict(gpu_lib, c, torch.zeros_like(w), 100, 3, 10)
    v = w.clone()
    v[..., ::3] = 0.0
    v[..., 1::3] = -0.0
    check_evict(gpu_lib, c, v, 200, 0, 0)
    v = w - 2
    v[..., ::5] = math.nan
    v[..., ::7] = math.inf
    v[..., ::11] = -math.inf
    for budget in (20, 150, 290):
        check_evict(gpu_lib, c, v, budget, 2, 5)
    check_evict(gpu_lib, c, torch.full_like(w, math.nan), 100, 3, 10)


def test_evict_lengths_and_pages_out_of_range(gpu_lib):
    lib = gpu_lib
    c, w = evict_case(2, 4, 2, 64, 16, (100, 200, 300, 50), BF, 21)
    c["ctx_len"] = torch.tensor([-1, 200, 303, 50], dtype=torch.int32)
    check_evict(lib, c, w, 64, 4, 4, error=lib.DEVERR_BAD_LENGTH)
    c, w = evict_case(2, 2, 2, 64, 16, (100, 200), BF, 22)
    c["page_table"][0, 3] = c["k_cache"].shape[1]
    c["page_table"][1, 0] = -1
    check_evict(lib, c, w, 64, 4, 4, error=lib.DEVERR_BAD_PAGE)


def test_evict_twice_and_in_a_graph(gpu_lib):
    """A second cut of a cut cache; a replay gives the eager call's bits."""
    lib = gpu_lib
    c, w = evict_case(2, 2, 2, 64, 16, (500, 800), BF, 23)
    t = {n: c[n].cuda() for n in ("k_cache", "v_cache", "page_table", "ctx_len")}
    wg = w.cuda()
    r = lib.ssd_kv_evict(t["k_cache"], t["v_cache"], t["page_table"], t["ctx_len"], wg, 300, sinks=2, recent=9)
    lib.ssd_kv_evict(t["k_cache"], t["v_cache"], t["page_table"], r["ctx_len"], r["weights"], 100, sinks=2, recent=9,
                     out={"weights": r["weights"]})
    k, v, new, kept, wout = cref.evict(c, w, 300, 2, 9)
    d = {**c, "k_cache": k, "v_cache": v, "ctx_len": new}
    k, v, new, kept, wout = cref.evict(d, wout, 100, 2, 9)
    torch.cuda.synchronize()
    assert torch.equal(t["k_cache"].cpu(), k) and torch.equal(t["v_cache"].cpu(), v)
    assert torch.equal(r["weights"].cpu(), wout)
    for n in ("k_cache", "v_cache"):
        t[n].copy_(c[n])
    ws, out = r["ws"], {}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    args = (t["k_cache"], t["v_cache"], t["page_table"], t["ctx_len"], wg, 100)
    lib.ssd_kv_evict(*args, ws=ws, out=out)  # (makes the outputs)
    for n in ("k_cache", "v_cache"):
        t[n].copy_(c[n])
    with torch.cuda.graph(g, stream=side):
        lib.ssd_kv_evict(*args, ws=ws, out=out)
    g.replay()
    torch.cuda.synchronize()
    k, v, new, kept, wout = cref.evict(c, w, 100)
    assert torch.equal(t["k_cache"].cpu(), k) and torch.equal(t["v_cache"].cpu(), v)
    assert torch.equal(out["kept"].cpu(), kept) and torch.equal(out["weights"].cpu(), wout)


# ---------------------------------------------------------------------------
# chains of more than 64 tokens, positions that are not slots
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("N,shift", [(70, None), (200, 1000), (3, 400)])
def test_append_of_chunks_and_positions(gpu_lib, N, shift):
    lib = gpu_lib
    c = case(2, N, 8, 2, 64, 16, (5, 130), BF, 24, packed=True, fill="random")
    c["cos_sin"] = lib.rope_table(4000, 64, device="cpu")
    c["n_nodes"] = torch.tensor([N, N - 1], dtype=torch.int32)
    g = ref.to_gpu(c)
    pos = None if shift is None else c["ctx_len"] + torch.tensor([shift, 2 * shift], dtype=torch.int32)
    r = lib.ssd_kv_append(g["q"], g["k"], g["v"], g["k_cache"], g["v_cache"], g["page_table"], g["ctx_len"],
                          n_nodes=g["n_nodes"], cos_sin=g["cos_sin"], pos=None if pos is None else pos.cuda())
    torch.cuda.synchronize()
    assert lib.get_device_error(r["ws"]) == 0
    kc, vc = c["k_cache"].double(), c["v_cache"].double()
    qo, kt, qt = torch.zeros(c["q"].shape, dtype=torch.float64), torch.zeros_like(kc), torch.zeros(c["q"].shape, dtype=torch.float64)
    for b in range(2):
        for j in range(N - b):
            at = int(c["ctx_len"][b]) + j if pos is None else int(pos[b]) + j
            cs, sn = c["cos_sin"][at, :32].double(), c["cos_sin"][at, 32:].double()

            def turn(x):
                x = x.double()
                a, z = x[..., :32], x[..., 32:]
                y = torch.cat([a * cs - z * sn, z * cs + a * sn], -1)
                return y, ref.HALF_STEP[BF] * y.abs() + 2.0 ** -19 * (a.abs() + z.abs()).repeat(1, 2)
            qo[b, j], qt[b, j] = turn(c["q"][b, j])
            p, o = ref.where(c, b, int(c["ctx_len"][b]) + j)
            kc[p, o], kt[p, o] = turn(c["k"][b, j])
            vc[p, o] = c["v"][b, j].double()
    _same(r["q"], qo, qt, "q")
    _same(g["k_cache"], kc, kt, "k_cache")
    assert torch.equal(g["v_cache"].double().cpu(), vc)
