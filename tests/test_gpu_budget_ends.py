"""Chunk attention, slot weights and eviction where they meet: waits that run out, streams and
graphs that share a workspace, windows of all sizes, and a run of the operators together."""
import math

import pytest
import torch

import chunk_reference as cref
import target_reference as ref
from test_gpu_budget import add_weights, check_evict, check_weights, evict_case
from test_gpu_chunk import attend, case, check
from test_gpu_target import _same
from test_gpu_waits import withheld  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("B,N,Hq,Hkv,D,ctx,dt", [
    (1, 1, 4, 1, 64, 900, BF),       # copies of rows, both warpgroups an item
    (3, 12, 16, 2, 128, 700, FP),    # one row tile
    (2, 8, 16, 2, 128, 5000, BF),    # copies, a warpgroup an item
    (2, 300, 8, 2, 64, 100, BF)])    # two row tiles
def test_tiles_that_do_not_arrive(gpu_lib, withheld, B, N, Hq, Hkv, D, ctx, dt):  # noqa: F811
    """The calls end with the error bit; then the same calls are right, with their workspaces."""
    lib = gpu_lib
    c = case(B, N, Hq, Hkv, D, 16, ctx, dt, 72)
    good = attend(lib, c)
    with withheld:
        attend(lib, c, ws=good["ws"])
    assert lib.get_device_error(good["ws"], clear=True) == lib.DEVERR_TIMEOUT
    again = attend(lib, c, ws=good["ws"])
    assert lib.get_device_error(good["ws"]) == 0
    assert torch.equal(again["out"], good["out"]) and torch.equal(again["lse"], good["lse"])
    lse, w = good["lse"].cpu(), torch.zeros((B, Hkv, ctx + N))
    first = add_weights(lib, c, lse, w)
    with withheld:
        add_weights(lib, c, lse, w, ws=first["ws"])
    assert lib.get_device_error(first["ws"], clear=True) == lib.DEVERR_TIMEOUT
    second = add_weights(lib, c, lse, w, ws=first["ws"])
    assert lib.get_device_error(first["ws"]) == 0
    assert torch.equal(first["weights"], second["weights"])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2 ** 31 - 1, 2 ** 31 - 1), (300, 2 ** 31 - 1), (8, 299),
                                          (1000, 7), (128, 128)])
def test_windows_of_all_sizes(gpu_lib, window, sinks):
    for N in (1, 40, 150):
        c = case(3, N, 8, 2, 64, 16, (0, 290, 131), BF, 30)
        check(gpu_lib, c, window, sinks)
        check_weights(gpu_lib, c, window, sinks, decay=0.5)


@pytest.mark.parametrize("G", [1, 3, 9, 16, 31, 64])
def test_groups_of_heads(gpu_lib, G):
    for N in (1, 2, 5, 64 // G + 1, 128 // G, 128 // G + 1):
        c = case(2, N, 2 * G, 2, 64, 16, (3, 260), FP, 31)
        check(gpu_lib, c, 200, 3)
        check_weights(gpu_lib, c, 200, 3)


def test_streams_and_graphs_that_share_a_workspace(gpu_lib):
    """Two graphs captured with one workspace, replayed in turn on a stream that is not the
    current one; the eager bits."""
    lib = gpu_lib
    cs = [ref.to_gpu(case(3, N, 8, 2, 128, 16, (40, 900, 333), BF, 32 + N)) for N in (2, 150)]
    at = [(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["ctx_len"]) for c in cs]
    want = [lib.ssd_chunk_attention(*x) for x in at]
    lse = [w["lse"] for w in want]
    ones = [torch.ones((3, 2, 1050), device="cuda") for _ in cs]
    sums = [lib.ssd_kv_weights(x[0], x[1], *x[3:], l, o.clone())["weights"] for x, l, o in zip(at, lse, ones)]
    ws = lib.new_workspace(max(lib.chunk_attention_workspace_bytes(3, c["q"].shape[1], 8, 2, 128) for c in cs) + 4096,
                           "cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs, got, graphs = [{}, {}], [o.clone() for o in ones], []
    wws = lib.ssd_kv_weights(at[0][0], at[0][1], *at[0][3:], lse[0], ones[0].clone())["ws"]
    torch.cuda.synchronize()
    for x, o, l, w in zip(at, outs, lse, got):
        lib.ssd_chunk_attention(*x, ws=ws, out=o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            lib.ssd_chunk_attention(*x, ws=ws, out=o)
            lib.ssd_kv_weights(x[0], x[1], *x[3:], l, w, ws=wws)
        graphs.append(g)
    for turn in range(3):
        for o, w in zip(outs, got):
            o["out"].fill_(math.nan)
            w.fill_(1.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for g in graphs if turn % 2 else graphs[::-1]:
                g.replay()
        side.synchronize()
        for o, w, r, s in zip(outs, got, want, sums):
            assert torch.equal(o["out"], r["out"]) and torch.equal(o["lse"], r["lse"]) and torch.equal(w, s)
    assert lib.get_device_error(ws) == 0 and lib.get_device_error(wws) == 0


def test_two_streams_at_once(gpu_lib):
    """Calls with workspaces of their own, one beside the other."""
    lib = gpu_lib
    cs = [ref.to_gpu(case(8, N, 8, 2, 64, 16, 700, BF, 40 + N)) for N in (1, 90)]
    at = [(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["ctx_len"]) for c in cs]
    want = [lib.ssd_chunk_attention(*x) for x in at]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(10):
        got = []
        for x, s, w in zip(at, streams, want):
            with torch.cuda.stream(s):
                got.append(lib.ssd_chunk_attention(*x, ws=w["ws"]))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g["out"], w["out"]) and torch.equal(g["lse"], w["lse"])


@pytest.mark.parametrize("D,order", [(64, "slot"), (128, "head")])
def test_a_budgeted_cache_from_prompt_to_decoding(gpu_lib, D, order):
    """Prompt chunks, weights of their last tokens, the cut, decoding at positions that are no
    slots any more, and a second cut: each step against its plain form on what the one before
    left on the GPU."""
    lib = gpu_lib
    B, Hq, Hkv, page, layers, S = 2, 8, 2, 16, 2, 400
    budget, sinks, recent = 90, 4, 20
    gen = torch.Generator().manual_seed(50)
    width = S // page
    shape = (layers, B * width, page, Hkv, D) if order == "slot" else (layers, B * width, Hkv, page, D)
    kv = [torch.zeros(shape, dtype=BF, device="cuda") for _ in range(2)]
    if order == "head":
        kv = [t.transpose(2, 3) for t in kv]
    table = torch.randperm(B * width, generator=gen).to(torch.int32).view(B, width)
    table_g = table.cuda()
    rope = lib.rope_table(1000, D, device="cpu")
    rope_g = rope.cuda()
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    weights = torch.zeros((layers, B, Hkv, S), device="cuda")
    tables = []

    def plain(layer, q):
        return {"N": q.shape[1], "page": page, "ctx_len": ctx.cpu(), "page_table": table, "q": q.cpu(),
                "k_cache": kv[0][layer].cpu(), "v_cache": kv[1][layer].cpu(), "parent": None, "n_nodes": None}

    def tokens(N, observers):
        nonlocal ctx, pos
        for layer in range(layers):
            x = torch.randn((B, N, Hq + 2 * Hkv, D), generator=gen).to(BF).cuda()
            q, k, v = x.split([Hq, Hkv, Hkv], 2)
            a = lib.ssd_kv_append(q, k, v, kv[0][layer], kv[1][layer], table_g, ctx, cos_sin=rope_g, pos=pos)
            at = int(ctx[1]) + N - 1  # the last key, turned by its position
            got = kv[0][layer][int(table[1, at // page]), at % page].double().cpu()
            p = int(pos[1]) + N - 1
            z = k[1, N - 1].double().cpu()
            cs, sn = rope[p, :D // 2].double(), rope[p, D // 2:].double()
            lo, hi = z[:, :D // 2], z[:, D // 2:]
            key = torch.cat([lo * cs - hi * sn, hi * cs + lo * sn], 1)
            size = (lo.abs() + hi.abs()).repeat(1, 2)
            assert bool(((got - key).abs() <= 2.0 ** -8 * key.abs() + 2.0 ** -19 * size).all())
            r = lib.ssd_chunk_attention(a["q"], kv[0][layer], kv[1][layer], table_g, ctx)
            c = plain(layer, a["q"])
            out, lse, tol, ltol = cref.attention(c)
            _same(r["out"], out, tol, "out")
            _same(r["lse"], lse, ltol, "lse")
            if observers:
                n = min(N, observers)
                l = r["lse"][:, N - n:].contiguous()
                before = weights[layer].cpu()
                u = lib.ssd_kv_weights(a["q"][:, N - n:], kv[0][layer], table_g, ctx + (N - n), l, weights[layer])
                c = {**c, "N": n, "q": c["q"][:, N - n:], "ctx_len": c["ctx_len"] + (N - n)}
                want, wtol = cref.weights(c, l.cpu(), before)
                _same(weights[layer], want, wtol, "weights")
                tables.append(u["ws"])
            tables.extend([a["ws"], r["ws"]])
        ctx, pos = ctx + N, pos + N

    def cut():
        nonlocal ctx
        c = {"ctx_len": ctx.cpu(), "page_table": table, "page": page, "k_cache": kv[0].cpu(), "v_cache": kv[1].cpu()}
        k, v, new, kept, wout = cref.evict(c, weights.cpu(), budget, sinks, recent)
        r = lib.ssd_kv_evict(kv[0], kv[1], table_g, ctx, weights, budget, sinks=sinks, recent=recent,
                             out={"weights": weights})
        assert torch.equal(kv[0].cpu(), k) and torch.equal(kv[1].cpu(), v)
        assert torch.equal(r["kept"].cpu(), kept) and torch.equal(weights.cpu(), wout)
        assert r["ctx_len"].tolist() == new.tolist() == [min(budget, int(x)) for x in ctx.tolist()]
        assert kept[0, 0, 0, :sinks].tolist() == list(range(sinks))
        ctx = r["ctx_len"]
        tables.append(r["ws"])

    tokens(130, 0)
    tokens(77, 32)
    cut()
    for _ in range(12):
        tokens(1, 1)
    tokens(6, 6)  # a drafted chain
    cut()
    tokens(1, 1)
    assert all(lib.get_device_error(w) == 0 for w in tables)


@pytest.mark.parametrize("ctx", [4094, 4500, 8190, 9000, 16500])
@pytest.mark.parametrize("layers,Hkv", [(1, 1), (5, 8), (19, 4), (19, 8), (20, 8)])
def test_cuts_of_all_numbers_of_heads(gpu_lib, layers, Hkv, ctx):
    """From one head to more than there are SMs, at lengths where the CTAs that choose a head's
    slots are one, two, four and eight."""
    if layers * Hkv > 100 and ctx > 5000:
        ctx = ctx // 4
    check_evict(gpu_lib, *evict_case(layers, 1, Hkv, 64, 16, ctx, BF, ctx), 700, 4, 100, in_place=Hkv == 4)


def test_batches_of_empty_sequences(gpu_lib):
    """No new tokens at all: zeros and -inf, the weights as they were; nothing to cut."""
    lib = gpu_lib
    for N, D in ((1, 64), (6, 128), (200, 64)):
        c = case(5, N, 8, 2, D, 16, (0, 40, 3, 0, 99), BF, 60, fill="random")
        c["n_nodes"] = torch.zeros(5, dtype=torch.int32)
        out = {"out": torch.full((5, N, 8, D), math.nan, dtype=BF, device="cuda"),
               "lse": torch.full((5, N, 8), math.nan, device="cuda")}
        r = attend(lib, c, out=out)
        assert bool((r["out"] == 0).all()) and bool((r["lse"] == -math.inf).all())
        w = torch.rand((5, 2, 300))
        u = add_weights(lib, c, torch.full((5, N, 8), -math.inf), w, decay=0.5)
        assert torch.equal(u["weights"].cpu(), w)
        assert lib.get_device_error(r["ws"]) == 0 and lib.get_device_error(u["ws"]) == 0
    check_evict(lib, *evict_case(2, 3, 2, 64, 16, (0, 0, 0), BF, 61), 7, 1, 2)


@pytest.mark.parametrize("N,D", [(1, 64), (2, 128)])
def test_many_sequences(gpu_lib, N, D):
    """More sequences than CTAs and than threads of one."""
    c = case(900, N, 4, 2, D, 16, tuple((i * 7) % 90 for i in range(900)), FP, 62, fill="random")
    check(gpu_lib, c, 50, 2)
    check_weights(gpu_lib, c, 50, 2)


@pytest.mark.parametrize("page", [16, 1])
def test_caches_beyond_32_bits(gpu_lib, page):
    """Pages behind the first 2^32 bytes and 2^31 entries of a cache."""
    lib = gpu_lib
    H, D = 8, 128
    small = case(2, 40, 16, H, D, page, (100, 333), BF, 70, fill="random")
    used = small["k_cache"].shape[0]
    first = (2 ** 31 + 2 ** 20) // (page * H * D)
    g = ref.to_gpu(small)
    for n in ("k_cache", "v_cache"):
        big = torch.empty((first + used, page, H, D), dtype=BF, device="cuda")
        big[first:] = g[n]
        g[n] = big
    g["page_table"] = torch.where(g["page_table"] >= 0, g["page_table"] + first, -1).to(torch.int32)
    out, lse, tol, ltol = cref.attention(small, 90, 3)
    r = lib.ssd_chunk_attention(g["q"], g["k_cache"], g["v_cache"], g["page_table"], g["ctx_len"], window=90, sinks=3)
    _same(r["out"], out, tol, "out")
    _same(r["lse"], lse, ltol, "lse")
    w = torch.rand((2, H, 400), generator=torch.Generator().manual_seed(2))
    want, wtol = cref.weights(small, r["lse"].cpu(), w, 90, 3)
    u = lib.ssd_kv_weights(g["q"], g["k_cache"], g["page_table"], g["ctx_len"], r["lse"], w.cuda(), window=90, sinks=3)
    _same(u["weights"], want, wtol, "weights")
    c = {**small, "k_cache": small["k_cache"][None], "v_cache": small["v_cache"][None]}
    k, v, new, kept, wout = cref.evict(c, w[None], 64, 4, 9)
    e = lib.ssd_kv_evict(g["k_cache"], g["v_cache"], g["page_table"], g["ctx_len"], w.cuda(), 64, sinks=4, recent=9)
    torch.cuda.synchronize()
    assert torch.equal(e["kept"].cpu(), kept[0]) and torch.equal(e["ctx_len"].cpu(), new)
    assert torch.equal(g["k_cache"][first:].cpu(), k[0]) and torch.equal(g["v_cache"][first:].cpu(), v[0])
    assert all(lib.get_device_error(x["ws"]) == 0 for x in (r, u, e))
