"""Attention of chunks over the paged cache against the plain form in 64 bits, at the sizes,
windows and values where it can go wrong.  Tolerances: tests/chunk_reference.py."""
import math

import pytest
import torch

import chunk_reference as cref
import target_reference as ref
from test_gpu_target import _same

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def case(B, N, Hq, Hkv, D, page, ctx, dtype, seed, ragged=False, order="slot", fill="nan", **kw):
    c = ref.case(B, N, Hq, Hkv, D, page, ctx, dtype, seed, tree="chain", order=order, **kw)
    if ragged:
        c["n_nodes"] = torch.tensor([(b * 7 + N) % (N + 1) for b in range(B)], dtype=torch.int32)
    if fill == "nan":  # every slot behind its sequence's end
        keep = torch.zeros(c["k_cache"].shape[:2], dtype=torch.bool)
        for b in range(B):
            s = torch.arange(int(c["ctx_len"][b]) + cref.tokens_of(c, b))
            keep[c["page_table"][b][s // page].long(), s % page] = True
        for t in (c["k_cache"], c["v_cache"]):
            t[~keep] = math.nan
    return c


def attend(lib, c, **kw):
    g = ref.to_gpu(c)
    r = lib.ssd_chunk_attention(g["q"], g["k_cache"], g["v_cache"], g["page_table"], g["ctx_len"],
                                n_nodes=g["n_nodes"], **kw)
    torch.cuda.synchronize()
    return r


def check(lib, c, window=0, sinks=0, scale=None, error=0):
    out, lse, tol, ltol = cref.attention(c, window, sinks, scale)
    r = attend(lib, c, window=window, sinks=sinks, scale=scale)
    assert lib.get_device_error(r["ws"]) == error
    _same(r["out"], out, tol, "out")
    _same(r["lse"], lse, ltol, "lse")
    return r


CASES = [
    # B, N, Hq, Hkv, D, page, ctx, dtype, ragged, order, window, sinks
    (1, 1, 1, 1, 128, 16, 0, BF, False, "slot", 0, 0),
    (1, 1, 4, 1, 64, 16, 1, FP, False, "slot", 1, 0),
    (2, 1, 8, 2, 128, 16, (127, 128), BF, False, "head", 0, 0),
    (3, 8, 8, 2, 128, 16, (120, 121, 500), BF, False, "slot", 0, 0),
    (3, 8, 8, 2, 128, 16, (120, 121, 500), BF, False, "slot", 100, 4),
    (2, 2, 16, 2, 64, 16, (700, 900), FP, False, "slot", 128, 16),
    (2, 16, 16, 2, 128, 16, (255, 900), BF, False, "slot", 17, 130),
    (2, 33, 4, 1, 128, 32, (0, 300), BF, True, "head", 0, 0),
    (1, 65, 2, 2, 64, 16, 0, BF, False, "slot", 0, 0),
    (1, 128, 1, 1, 128, 16, 0, FP, False, "slot", 0, 0),
    (1, 257, 1, 1, 128, 16, 3, BF, False, "slot", 0, 0),
    (1, 300, 5, 1, 64, 16, 77, FP, False, "slot", 0, 0),
    (1, 300, 5, 1, 64, 16, 77, FP, False, "slot", 64, 3),
    (2, 140, 14, 2, 128, 64, (0, 129), BF, True, "slot", 0, 0),
    (2, 140, 14, 2, 128, 64, (0, 1290), BF, True, "slot", 256, 64),
    (1, 70, 12, 1, 128, 128, 250, BF, False, "head", 0, 0),
    (1, 9, 64, 1, 64, 16, 130, BF, False, "slot", 0, 0),
    (1, 5, 48, 1, 128, 16, 90, FP, False, "slot", 50, 1),
    (2, 40, 6, 3, 64, 1, (30, 45), BF, False, "slot", 20, 2),
    (2, 70, 4, 2, 128, 5, (61, 300), FP, False, "head", 0, 0),
    (2, 70, 4, 2, 128, 5, (61, 300), BF, False, "slot", 90, 7),
    (2, 12, 4, 4, 128, 24, (119, 121), BF, False, "slot", 0, 0),
    (2, 90, 4, 2, 64, 200, (190, 401), BF, False, "slot", 130, 10),
    (2, 90, 4, 2, 64, 200, (190, 401), BF, False, "head", 0, 0),
    (1, 30, 4, 2, 128, 256, 300, FP, False, "head", 0, 0),
    (1, 200, 4, 2, 128, 256, 700, FP, False, "slot", 300, 260),
    (70, 2, 4, 2, 64, 16, tuple((i * 37) % 211 for i in range(70)), BF, True, "slot", 0, 0),
    (70, 1, 8, 2, 128, 16, tuple((i * 371) % 1211 for i in range(70)), BF, False, "slot", 200, 4),
    (1, 8, 8, 1, 128, 16, 6000, BF, False, "slot", 0, 0),
    (1, 64, 8, 1, 128, 16, 5000, BF, False, "slot", 0, 0),
    (20, 40, 16, 4, 64, 32, tuple((i * 131) % 1500 for i in range(20)), FP, True, "slot", 0, 0),
    (20, 40, 16, 4, 128, 32, tuple((i * 131) % 1500 for i in range(20)), BF, True, "slot", 100, 100),
    (1, 700, 8, 2, 128, 16, 0, BF, False, "slot", 0, 0),
    (1, 700, 8, 2, 64, 16, 513, BF, False, "slot", 333, 5),
    (3, 500, 2, 2, 128, 48, (0, 1000, 100), FP, True, "slot", 0, 0),
    (1, 600, 1, 1, 64, 16, 100, BF, False, "slot", 150, 0),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(x) for x in c[:6] + c[10:]))
def test_chunk_attention(gpu_lib, c):
    B, N, Hq, Hkv, D, page, ctx, dt, ragged, order, window, sinks = c
    check(gpu_lib, case(B, N, Hq, Hkv, D, page, ctx, dt, 300 + N, ragged, order, width_extra=1), window, sinks)


@pytest.mark.parametrize("scale", [0.3, -0.05, 0.0])
def test_packed_queries_and_scale(gpu_lib, scale):
    for N in (6, 150):
        c = case(3, N, 8, 2, 128, 16, (5, 90, 200), BF, 7, packed=True)
        assert not c["q"].is_contiguous()
        check(gpu_lib, c, scale=scale)
        check(gpu_lib, c, scale=scale, window=40, sinks=8)


def test_rising_scores(gpu_lib):
    """Scores that grow along the context (the running maximum moves in every tile) and ones
    that fall (it never does)."""
    for sign in (1.0, -1.0):
        for N in (4, 200):
            c = case(2, N, 4, 2, 64, 16, (900, 1030), BF, 8, fill="random")
            c["q"] = torch.ones_like(c["q"])
            for b in range(2):
                s = torch.arange(int(c["ctx_len"][b]) + N)
                k = (sign * s.float() * 0.125 / 8).to(BF)[:, None, None].expand(-1, 2, 64)
                c["k_cache"][c["page_table"][b][s // 16].long(), s % 16] = k
            check(gpu_lib, c)


@pytest.mark.parametrize("window", [0, 30])
def test_unseen_values_do_not_leak(gpu_lib, window):
    """A token that holds NaN or infinities spoils those that see it, nobody else."""
    for N, ctx in ((16, (40, 133)), (150, (0, 200))):
        c = case(2, N, 8, 2, 128, 16, ctx, BF, 9)
        for b in range(2):
            L = int(c["ctx_len"][b])
            p, o = ref.where(c, b, L + 9)
            c["k_cache"][p, o] = math.nan
            c["v_cache"][p, o] = math.nan
            p, o = ref.where(c, b, L + 5)
            c["v_cache"][p, o, :, 3] = math.inf
            c["v_cache"][p, o, :, 9] = -math.inf
            p, o = ref.where(c, b, L // 2 + 1)
            c["v_cache"][p, o, 1, 70] = math.inf
        check(gpu_lib, c, window, 2 if window else 0)


def test_infinite_scores(gpu_lib):
    """A key of -inf against a positive query scores -inf: no weight; a row with nothing else
    is empty."""
    c = case(1, 2, 2, 1, 64, 16, 3, BF, 10)
    c["q"] = c["q"].abs() + 0.5
    for s in range(5):
        p, o = ref.where(c, 0, s)
        c["k_cache"][p, o] = -math.inf
    r = attend(gpu_lib, c)
    assert torch.equal(r["out"], torch.zeros_like(r["out"])) and bool((r["lse"] == -math.inf).all())
    p, o = ref.where(c, 0, 1)
    c["k_cache"][p, o] = 0.25
    r = attend(gpu_lib, c)
    assert torch.equal(r["out"].cpu(), c["v_cache"][p, o].expand(1, 2, 2, 64))


def test_lengths_and_pages_out_of_range(gpu_lib):
    lib = gpu_lib
    c = case(5, 70, 4, 2, 128, 16, (20, 33, 50, 7, 9), BF, 11, ragged=True, fill="random")
    c["ctx_len"][0] = -1
    c["ctx_len"][1] = 16 * c["page_table"].shape[1] - 2
    c["n_nodes"] = torch.tensor([70, 70, 71, -1, 60], dtype=torch.int32)
    check(lib, c, error=lib.DEVERR_BAD_LENGTH)
    c = case(2, 70, 4, 2, 128, 16, (40, 100), BF, 12, fill="random")
    c["page_table"][0, 1] = c["k_cache"].shape[0]
    c["page_table"][1, 4] = -3
    check(lib, c, error=lib.DEVERR_BAD_PAGE)
    check(lib, c, window=20, sinks=3, error=lib.DEVERR_BAD_PAGE)


def test_padded_batch_rows_and_empty_sequences(gpu_lib):
    """Tokens behind a sequence's last get zeros; nothing else of `out` is touched."""
    c = case(3, 130, 4, 2, 64, 16, (0, 64, 30), BF, 13, fill="random")
    c["n_nodes"] = torch.tensor([0, 1, 129], dtype=torch.int32)
    out = {"out": torch.full((3, 130, 4, 64), math.nan, dtype=BF, device="cuda"),
           "lse": torch.full((3, 130, 4), math.nan, device="cuda")}
    want, lse, tol, ltol = cref.attention(c)
    r = attend(gpu_lib, c, out=out)
    _same(r["out"], want, tol, "out")
    _same(r["lse"], lse, ltol, "lse")


@pytest.mark.parametrize("dt", [BF, FP])
def test_values_of_all_sizes(gpu_lib, dt):
    """Finite results for finite values up to the type's largest, and no loss for small ones."""
    big = torch.finfo(dt).max
    for N in (3, 200):
        for f in (big, 1e-20 if dt == BF else 6e-5):
            c = case(1, N, 8, 2, 64, 16, 900, dt, 14)
            c["v_cache"] = (c["v_cache"].sign() * f).to(dt)
            check(gpu_lib, c)


def test_same_bits_every_call_and_in_a_graph(gpu_lib):
    """Replays with other lengths in the same tensors; the eager call's bits."""
    lib = gpu_lib
    for N, window in ((1, 64), (200, 0)):
        c = ref.to_gpu(case(6, N, 8, 2, 128, 16, tuple(100 + 150 * i for i in range(6)), BF, 15, fill="random",
                            width_extra=8))
        n = torch.full((6,), N, dtype=torch.int32, device="cuda")
        args = (c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["ctx_len"])
        out, kw = {}, dict(n_nodes=n, window=window, sinks=4)
        r = lib.ssd_chunk_attention(*args, **kw, out=out)
        ws = r["ws"]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            lib.ssd_chunk_attention(*args, **kw, ws=ws, out=out)
        for lens in (c["ctx_len"].clone(), c["ctx_len"] // 2, c["ctx_len"] * 0 + 3):
            c["ctx_len"].copy_(lens)
            n.copy_(torch.tensor([N, 0, N, max(0, N - 1), 1, N], dtype=torch.int32))
            g.replay()
            torch.cuda.synchronize()
            first = (out["out"].clone(), out["lse"].clone())
            r = lib.ssd_chunk_attention(*args, **kw)
            assert torch.equal(r["out"], first[0]) and torch.equal(r["lse"], first[1])
            assert lib.get_device_error(ws) == 0


@pytest.mark.parametrize("N", [1, 24, 200])
def test_nothing_of_an_earlier_kernel_stays_in_shared_memory(gpu_lib, N):
    """Pages of 5: the rows between them, in tiles of which the window leaves few pages, after a
    call that filled every CTA's shared memory with NaN."""
    c = case(8, N, 20, 4, 128, 16, 3000, FP, 16, fill="random")
    c["v_cache"][:] = math.nan
    c["k_cache"][:] = math.nan
    attend(gpu_lib, c)
    check(gpu_lib, case(22, N, 20, 4, 128, 5, tuple(i * 61 for i in range(22)), FP, 17, order="head"), 128, 1)


@pytest.mark.parametrize("page", [2, 12, 40, 72, 130, 136, 201])
def test_page_sizes(gpu_lib, page):
    """Pages whose parts make a tile, ones that need whole pages, and both kinds above 128."""
    for N, D, order in ((1, 64, "slot"), (60, 128, "slot"), (60, 128, "head"), (210, 64, "slot")):
        c = case(3, N, 8, 2, D, page, (0, 131, 620), BF, page, order=order)
        check(gpu_lib, c)
        check(gpu_lib, c, 150, 9)


@pytest.mark.parametrize("page", [1, 3, 5, 12, 130, 201])
@pytest.mark.parametrize("gap", [False, True])
def test_odd_pages_out_of_range_and_apart(gpu_lib, page, gap):
    """Page ids out of range give zeros; the same with pages that lie no whole number of slots
    apart (and after a call that left NaN in shared memory)."""
    lib = gpu_lib
    for N, D in ((1, 64), (50, 128), (200, 64)):
        if gap:
            nans = case(8, N, 8, 2, D, 16, 3000, BF, 16, fill="random")
            nans["v_cache"][:] = math.nan
            nans["k_cache"][:] = math.nan
            attend(lib, nans)
        c = case(2, N, 8, 2, D, page, (150, 420), BF, 60 + page, fill="random")
        if gap:
            for n in ("k_cache", "v_cache"):
                t = c[n]
                flat = torch.zeros((t.shape[0], page * 2 * D + 8), dtype=BF, device="cuda")
                c[n] = flat[:, :page * 2 * D].view(t.shape)
                c[n].copy_(t)
        g = ref.to_gpu({**c, "k_cache": None, "v_cache": None})
        for bad in (False, True):
            if bad:
                c["page_table"][0, 100 // page] = c["k_cache"].shape[0]
                c["page_table"][1, 300 // page] = -2
                g["page_table"] = c["page_table"].cuda()
            plain = {**c, "k_cache": c["k_cache"].cpu(), "v_cache": c["v_cache"].cpu()}
            for window, sinks in ((0, 0), (330, 2)):
                out, lse, tol, ltol = cref.attention(plain, window, sinks)
                r = lib.ssd_chunk_attention(g["q"], c["k_cache"].cuda() if not gap else c["k_cache"],
                                            c["v_cache"].cuda() if not gap else c["v_cache"], g["page_table"],
                                            g["ctx_len"], window=window, sinks=sinks)
                torch.cuda.synchronize()
                assert lib.get_device_error(r["ws"]) == (lib.DEVERR_BAD_PAGE if bad else 0)
                _same(r["out"], out, tol, "out")
                _same(r["lse"], lse, ltol, "lse")
