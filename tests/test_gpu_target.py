"""The target pass's operators (paged-cache append, tree attention, commit of
the accepted path, token log probabilities) against their plain forms in 64
bits, at the sizes and masks where they can go wrong.

Tolerances: a rounding to 16 bits is off by at most half a step of the value;
what happens in 32 bits is bounded in tests/target_reference.py.
"""
import math

import pytest
import torch

import target_reference as ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def _attend(lib, c, **kw):
    g = ref.to_gpu(c)
    r = lib.ssd_tree_attention(g["q"], g["k_cache"], g["v_cache"], g["page_table"], g["ctx_len"],
                               parent=g["parent"], n_nodes=g["n_nodes"], **kw)
    torch.cuda.synchronize()
    return r


def _same(got, want, tol, what):
    got, want = got.double().cpu(), want
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN elsewhere"
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf]), what + ": infinities"
    fine = torch.isfinite(want)
    over = ((got - want).abs() - tol)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, "%s: %d entries beyond, by up to %.3g" % (
        what, int((over > 0).sum()), float(over.max()))


def _check_attention(lib, c, **kw):
    out, lse, tol, ltol = ref.attention(c, kw.get("scale"))
    r = _attend(lib, c, **kw)
    _same(r["out"], out, tol, "out")
    _same(r["lse"], lse, ltol, "lse")
    return r


ATTN = [
    # B, N, Hq, Hkv, D, page, ctx, dtype, tree, ragged, order
    (1, 1, 1, 1, 128, 16, 0, BF, "chain", False, "slot"),
    (1, 1, 4, 1, 64, 16, 1, FP, "chain", False, "slot"),
    (2, 1, 8, 2, 128, 16, (127, 128), BF, "chain", False, "head"),
    (3, 8, 8, 2, 128, 16, (120, 121, 500), BF, "chain", False, "slot"),
    (3, 8, 32, 4, 128, 16, (0, 250, 1000), FP, "random", False, "slot"),
    (2, 21, 16, 2, 128, 16, (235, 300), BF, "random", False, "head"),
    (2, 21, 14, 2, 64, 32, (107, 640), BF, "random", True, "slot"),
    (2, 64, 4, 1, 128, 64, (64, 700), BF, "random", False, "slot"),
    (1, 64, 12, 1, 64, 16, 257, FP, "random", False, "slot"),
    (4, 33, 10, 2, 128, 128, (0, 1, 95, 96), BF, "random", True, "head"),
    (2, 5, 6, 3, 64, 1, (30, 45), BF, "random", False, "slot"),
    (2, 7, 4, 2, 128, 5, (61, 300), FP, "random", False, "head"),
    (2, 12, 4, 4, 128, 24, (119, 121), BF, "random", False, "slot"),
    (2, 9, 4, 2, 64, 200, (190, 401), BF, "random", False, "slot"),
    (1, 3, 4, 2, 128, 256, 300, FP, "chain", False, "head"),
    (70, 2, 4, 2, 64, 16, tuple((i * 37) % 211 for i in range(70)), BF, "random", True, "slot"),
    (1, 8, 8, 1, 128, 16, 6000, BF, "random", False, "slot"),
    (1, 64, 5, 1, 128, 16, 1500, BF, "random", False, "slot"),
    (1, 64, 64, 1, 64, 16, 130, BF, "random", False, "slot"),
    # several (sequence, head)s and tiles a CTA: 32, 64, 104, 168 and 256 rows
    (60, 2, 64, 4, 64, 16, tuple(100 + (i * 131) % 1500 for i in range(60)), FP, "chain", False, "slot"),
    (40, 8, 32, 4, 128, 16, tuple((i * 131) % 1500 for i in range(40)), BF, "random", True, "slot"),
    (40, 13, 32, 4, 128, 32, tuple((i * 131) % 1500 for i in range(40)), BF, "random", False, "head"),
    (24, 21, 32, 4, 128, 16, tuple((i * 231) % 2500 for i in range(24)), BF, "random", False, "slot"),
    (10, 64, 16, 4, 64, 16, tuple((i * 431) % 3500 for i in range(10)), FP, "random", True, "slot"),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(x) for x in c[:6]))
def test_tree_attention(gpu_lib, case):
    B, N, Hq, Hkv, D, page, ctx, dt, tree, ragged, order = case
    c = ref.case(B, N, Hq, Hkv, D, page, ctx, dt, 100 + N, tree, ragged, order, fill="nan", width_extra=1)
    _check_attention(gpu_lib, c)


def test_attention_packed_queries_and_scale(gpu_lib):
    c = ref.case(3, 6, 8, 2, 128, 16, (5, 90, 200), BF, 7, packed=True)
    assert not c["q"].is_contiguous()
    _check_attention(gpu_lib, c, scale=0.3)
    _check_attention(gpu_lib, c, scale=-0.05)
    _check_attention(gpu_lib, c, scale=0.0)


def test_attention_rising_scores(gpu_lib):
    """Scores that grow along the context (the running maximum moves in every
    tile) and ones that fall (it never does)."""
    for sign in (1.0, -1.0):
        c = ref.case(2, 4, 4, 2, 64, 16, (900, 1030), BF, 8)
        c["q"] = torch.ones_like(c["q"])
        ramp = torch.arange(c["page_table"].shape[1] * 16).float()
        for b in range(2):
            for s in range(int(c["ctx_len"][b]) + 4):
                p, o = ref.where(c, b, s)
                c["k_cache"][p, o] = (sign * ramp[s] * 0.125 * torch.ones(64) / 8).to(BF)
        _check_attention(gpu_lib, c)


def test_attention_unseen_values_do_not_leak(gpu_lib):
    """A node that holds NaN or infinities spoils those that see it, nobody
    else; an infinite value stays infinite where it is seen."""
    c = ref.case(2, 16, 8, 2, 128, 16, (40, 133), BF, 9)
    par = [-1, 0, 0, 1, 1, 2, 2, 3, 3, 4, 4, 5, 5, 6, 6, 7]
    c["parent"] = torch.tensor([par, par], dtype=torch.int32)
    for b in range(2):
        L = int(c["ctx_len"][b])
        p, o = ref.where(c, b, L + 3)
        c["k_cache"][p, o] = math.nan
        c["v_cache"][p, o] = math.nan
        p, o = ref.where(c, b, L + 5)
        c["v_cache"][p, o, :, 3] = math.inf
        c["v_cache"][p, o, :, 9] = -math.inf
    _check_attention(gpu_lib, c)


def test_attention_infinite_scores(gpu_lib):
    """A key of -inf against a positive query scores -inf: no weight; a row
    with nothing else is empty."""
    c = ref.case(1, 2, 2, 1, 64, 16, 3, BF, 10, tree="chain")
    c["q"] = c["q"].abs() + 0.5
    for s in range(5):
        p, o = ref.where(c, 0, s)
        c["k_cache"][p, o] = -math.inf
    r = _attend(gpu_lib, c)
    assert torch.equal(r["out"], torch.zeros_like(r["out"])) and bool((r["lse"] == -math.inf).all())
    p, o = ref.where(c, 0, 1)
    c["k_cache"][p, o] = 0.25
    r = _attend(gpu_lib, c)
    assert torch.equal(r["out"].cpu(), c["v_cache"][p, o].expand(1, 2, 2, 64))


def test_attention_absent_nodes(gpu_lib):
    c = ref.case(5, 6, 4, 2, 128, 16, (20, 33, 50, 7, 9), BF, 11)
    c["parent"][0] = torch.tensor([-1, 0, 3, 1, 2, 0])    # node 2 points ahead: 2 and 4 absent
    c["parent"][1] = torch.tensor([0, 0, 0, 0, 0, 0])     # no root: the walk of every node is broken
    c["n_nodes"] = torch.tensor([6, 6, 0, 3, 7], dtype=torch.int32)  # 7 > N
    r = _check_attention(gpu_lib, c)
    o = r["out"].cpu()
    assert not o[1].any() and not o[2].any() and not o[4].any() and not o[0, 2].any() and not o[0, 4].any()
    assert gpu_lib.get_device_error(r["ws"], clear=True) == (
        gpu_lib.DEVERR_BAD_TREE | gpu_lib.DEVERR_BAD_LENGTH)
    c["ctx_len"] = torch.tensor([-1, 20, 1 << 30, 0, 0], dtype=torch.int32)
    c["n_nodes"] = None
    c["parent"] = None
    _check_attention(gpu_lib, c)


def test_attention_bad_pages(gpu_lib):
    c = ref.case(3, 4, 4, 2, 64, 16, (60, 61, 100), BF, 12)
    c["page_table"][0, 1] = -1
    c["page_table"][2, 0] = c["k_cache"].shape[0]
    r = _check_attention(gpu_lib, c)
    assert gpu_lib.get_device_error(r["ws"], clear=True) == gpu_lib.DEVERR_BAD_PAGE
    assert gpu_lib.get_device_error(r["ws"]) == 0


def test_attention_far_pages(gpu_lib):
    """Pages whose entries lie beyond 2^32 elements."""
    pages = 36000
    kc, vc = (torch.empty((pages, 16, 64, 128), dtype=BF, device="cuda") for _ in range(2))
    assert kc.numel() > 1 << 32
    c = ref.case(1, 4, 64, 64, 128, 16, 40, BF, 13)
    want, lse, tol, ltol = ref.attention(c)
    table = torch.tensor([[pages - 1, 5, pages - 2]], dtype=torch.int32, device="cuda")
    for i in range(3):
        p = int(c["page_table"][0, i])
        kc[int(table[0, i])] = c["k_cache"][p].cuda()
        vc[int(table[0, i])] = c["v_cache"][p].cuda()
    g = ref.to_gpu(c)
    r = gpu_lib.ssd_tree_attention(g["q"], kc, vc, table, g["ctx_len"], parent=g["parent"])
    _same(r["out"], want, tol, "out")
    # the same far slots written by the append and moved by the commit
    r = gpu_lib.ssd_kv_append(g["q"], g["k"], g["v"], kc, vc, table, g["ctx_len"], parent=g["parent"])
    for j in range(4):
        page, o = int(table[0, (40 + j) // 16]), (40 + j) % 16
        assert torch.equal(kc[page, o], g["k"][0, j]) and torch.equal(vc[page, o], g["v"][0, j])
    node = torch.tensor([[3, -1, -1, -1]], dtype=torch.int32, device="cuda")
    one = torch.tensor([1], dtype=torch.int32, device="cuda")
    gpu_lib.ssd_kv_commit(kc, vc, table, g["ctx_len"], one, node)
    assert torch.equal(kc[pages - 2, 9], g["k"][0, 3]) and torch.equal(vc[pages - 2, 9], g["v"][0, 3])


def test_attention_repeats_streams_graph(gpu_lib):
    """The same bits from every run, on another stream, from a graph, and with
    a workspace that other sizes used in between."""
    c = ref.case(3, 21, 16, 2, 128, 16, (700, 100, 2000), BF, 14)
    d = ref.case(2, 2, 4, 2, 64, 16, (50, 9), FP, 15)
    g, h = ref.to_gpu(c), ref.to_gpu(d)
    n = max(gpu_lib.tree_attention_workspace_bytes(3, 21, 16, 2, 128),
            gpu_lib.tree_attention_workspace_bytes(2, 2, 4, 2, 64))
    ws = gpu_lib.new_workspace(n, "cuda")

    def run(x, **kw):
        return gpu_lib.ssd_tree_attention(x["q"], x["k_cache"], x["v_cache"], x["page_table"],
                                          x["ctx_len"], parent=x["parent"], ws=ws, **kw)
    a = run(g)
    first = a["out"].clone(), a["lse"].clone()
    run(h)
    b = run(g)
    assert torch.equal(b["out"], first[0]) and torch.equal(b["lse"], first[1])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = {"out": torch.empty_like(first[0]), "lse": torch.empty_like(first[1])}
    run(g, stream=s, out=out)
    s.synchronize()
    assert torch.equal(out["out"], first[0])
    graph = torch.cuda.CUDAGraph()
    out["out"].zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(g, out=out)
    g["ctx_len"].copy_(torch.tensor([650, 90, 1900], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    c["ctx_len"] = g["ctx_len"].cpu()
    want, lse, tol, ltol = ref.attention(c)
    _same(out["out"], want, tol, "out after a change of lengths")


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
APPEND = [
    # B, N, Hq, Hkv, D, page, ctx, dtype, tree, ragged, order, rot, interleaved, norm, packed
    (1, 1, 1, 1, 128, 16, 0, BF, "chain", False, "slot", 128, False, True, False),
    (1, 8, 64, 8, 128, 16, 100, BF, "chain", False, "slot", 128, False, True, True),
    (3, 5, 6, 3, 64, 5, (0, 3, 44), FP, "random", True, "head", 64, False, False, True),
    (2, 21, 7, 1, 128, 16, (9, 31), BF, "random", False, "slot", 32, True, True, True),
    (2, 64, 5, 5, 64, 24, (1, 130), FP, "random", False, "head", 48, False, True, False),
    (4, 3, 2, 1, 128, 1, (0, 1, 2, 9), BF, "random", False, "slot", 96, False, False, True),
    (2, 4, 12, 2, 128, 32, (10, 60), BF, "random", True, "slot", 0, False, False, True),
    (150, 6, 9, 3, 64, 16, tuple(i % 90 for i in range(150)), BF, "random", True, "slot", 64, True, True, True),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c[:6] + c[11:]))
def test_kv_append(gpu_lib, case):
    B, N, Hq, Hkv, D, page, ctx, dt, tree, ragged, order, rot, inter, norm, packed = case
    c = ref.case(B, N, Hq, Hkv, D, page, ctx, dt, 200 + N, tree, ragged, order, packed=packed)
    gen = torch.Generator().manual_seed(3)
    if rot:
        c["cos_sin"] = gpu_lib.rope_table(int(c["ctx_len"].max()) + N, rot, device="cpu")
    if norm:
        c["q_norm"], c["k_norm"] = ((torch.rand(D, generator=gen) + 0.5).to(dt) for _ in range(2))
    q, kc, vc, qt, kt = ref.append(c, rot, inter, 1e-5)
    g = ref.to_gpu(c)
    r = gpu_lib.ssd_kv_append(g["q"], g["k"], g["v"], g["k_cache"], g["v_cache"], g["page_table"],
                              g["ctx_len"], parent=g["parent"], n_nodes=g["n_nodes"],
                              cos_sin=g.get("cos_sin"), interleaved=inter, q_norm=g.get("q_norm"),
                              k_norm=g.get("k_norm"), eps=1e-5)
    _same(r["q"], q, qt, "q")
    _same(g["k_cache"], kc, kt, "k_cache")
    assert torch.equal(g["v_cache"].cpu().double(), vc)
    assert gpu_lib.get_device_error(r["ws"]) == 0


def test_kv_append_in_place_and_unaligned(gpu_lib):
    c = ref.case(2, 5, 6, 2, 128, 16, (3, 40), BF, 21)
    c["cos_sin"] = gpu_lib.rope_table(64, 128, device="cpu")
    q, kc, vc, qt, kt = ref.append(c, 128)
    g = ref.to_gpu(c)
    args = (g["k_cache"], g["v_cache"], g["page_table"], g["ctx_len"])
    r = gpu_lib.ssd_kv_append(g["q"], g["k"], g["v"], *args, parent=g["parent"], cos_sin=g["cos_sin"],
                              out={"q": g["q"]})
    assert r["q"].data_ptr() == g["q"].data_ptr()
    _same(r["q"], q, qt, "q in place")
    # a projection whose rows start at odd elements
    wide = torch.zeros((2, 5, 10 * 128 + 3), dtype=BF, device="cuda")
    view = wide[:, :, 1:1 + 1280].unflatten(2, (10, 128))
    h = ref.to_gpu(c)
    view[:, :, :6], view[:, :, 6:8], view[:, :, 8:] = h["q"], h["k"], h["v"]
    r = gpu_lib.ssd_kv_append(view[:, :, :6], view[:, :, 6:8], view[:, :, 8:], h["k_cache"], h["v_cache"],
                              h["page_table"], h["ctx_len"], parent=h["parent"], cos_sin=h["cos_sin"])
    _same(r["q"], q, qt, "q unaligned")
    _same(h["k_cache"], kc, kt, "k unaligned")


def test_kv_append_absent_nodes(gpu_lib):
    c = ref.case(5, 4, 4, 2, 64, 16, (20, 33, 50, 7, 9), BF, 22)
    c["parent"][0] = torch.tensor([-1, 2, 0, 1])
    c["n_nodes"] = torch.tensor([4, -1, 0, 3, 4], dtype=torch.int32)
    c["page_table"][4, 0] = 999
    c["cos_sin"] = gpu_lib.rope_table(52, 64, device="cpu")
    c["ctx_len"][3] = 51   # positions 51 .. : only the root's fits the table
    c["page_table"][3] = c["page_table"][2]
    q, kc, vc, qt, kt = ref.append(c, 64)
    g = ref.to_gpu(c)
    r = gpu_lib.ssd_kv_append(g["q"], g["k"], g["v"], g["k_cache"], g["v_cache"], g["page_table"],
                              g["ctx_len"], parent=g["parent"], n_nodes=g["n_nodes"], cos_sin=g["cos_sin"])
    _same(r["q"], q, qt, "q")
    _same(g["k_cache"], kc, kt, "k_cache")
    assert gpu_lib.get_device_error(r["ws"]) == (
        gpu_lib.DEVERR_BAD_TREE | gpu_lib.DEVERR_BAD_LENGTH | gpu_lib.DEVERR_BAD_PAGE)


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layers,B,N,H,D,page,order", [
    (1, 1, 1, 1, 64, 16, "slot"), (3, 4, 21, 2, 128, 16, "slot"), (2, 9, 64, 3, 64, 5, "head"),
    (5, 70, 13, 1, 128, 1, "slot")])
def test_kv_commit(gpu_lib, layers, B, N, H, D, page, order):
    gen = torch.Generator().manual_seed(30 + N)
    c = ref.case(B, N, H, H, D, page, [(b * 13) % 70 for b in range(B)], BF, 31, order=order)
    k, v = (torch.stack([t] + [torch.randn(t.shape, generator=gen).to(BF) for _ in range(layers - 1)])
            for t in (c["k_cache"], c["v_cache"]))
    node = torch.full((B, N), -1, dtype=torch.int32)
    acc = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        m = int(torch.randint(0, N, (), generator=gen))
        path = sorted((torch.randperm(N - 1, generator=gen)[:m] + 1).tolist()) if N > 1 else []
        if b == 1:
            path = list(range(1, N))     # nothing to move
        if b == 2:
            path = [N - 1]
        acc[b], node[b, :len(path)] = len(path), torch.tensor(path, dtype=torch.int32)
    if B > 3:
        acc[3] = -2
    kw, vw = k.clone(), v.clone()
    for b in range(B):
        L = int(c["ctx_len"][b])
        for i in range(max(0, int(acc[b]))):
            (p0, o0), (p1, o1) = ref.where(c, b, L + int(node[b, i])), ref.where(c, b, L + 1 + i)
            kw[:, p1, o1], vw[:, p1, o1] = k[:, p0, o0], v[:, p0, o0]
    if order == "head":
        kg, vg = (t.transpose(2, 3).contiguous().cuda().transpose(2, 3) for t in (k, v))
    else:
        kg, vg = k.cuda(), v.cuda()
    r = gpu_lib.ssd_kv_commit(kg, vg, c["page_table"].cuda(), c["ctx_len"].cuda(), acc.cuda(), node.cuda())
    assert torch.equal(kg.cpu(), kw) and torch.equal(vg.cpu(), vw)
    want = torch.where(acc < 0, c["ctx_len"], c["ctx_len"] + 1 + acc)
    assert torch.equal(r["ctx_len"].cpu(), want)
    assert gpu_lib.get_device_error(r["ws"]) == 0
    r = gpu_lib.ssd_kv_commit(kg, vg, c["page_table"].cuda(), c["ctx_len"].cuda(), acc.cuda())
    assert torch.equal(kg.cpu(), kw) and torch.equal(r["ctx_len"].cpu(), want)  # a chain moves nothing


def test_kv_commit_refused_rows(gpu_lib):
    """Paths that are none, lengths and pages out of range: nothing moves."""
    c = ref.case(6, 5, 2, 2, 64, 8, (4, 4, 4, 4, 4, 4), BF, 32)
    node = torch.tensor([[2, 2, -1, -1, -1], [5, -1, -1, -1, -1], [0, -1, -1, -1, -1],
                         [3, 1, -1, -1, -1], [2, 4, -1, -1, -1], [2, 3, -1, -1, -1]], dtype=torch.int32)
    acc = torch.tensor([2, 1, 1, 2, 2, 2], dtype=torch.int32)
    ctx = c["ctx_len"].clone()
    ctx[4] = 1000
    c["page_table"][5] = -1
    g = ref.to_gpu(c)
    r = gpu_lib.ssd_kv_commit(g["k_cache"], g["v_cache"], g["page_table"], ctx.cuda(), acc.cuda(), node.cuda())
    assert torch.equal(g["k_cache"].cpu(), c["k_cache"]) and torch.equal(g["v_cache"].cpu(), c["v_cache"])
    assert r["ctx_len"].tolist() == [4, 4, 4, 4, 1000, 7]
    assert gpu_lib.get_device_error(r["ws"]) == (
        gpu_lib.DEVERR_BAD_TREE | gpu_lib.DEVERR_BAD_LENGTH | gpu_lib.DEVERR_BAD_PAGE)


# ---------------------------------------------------------------------------
# log probabilities
# ---------------------------------------------------------------------------
def _check_logprobs(lib, z, tok, K, T=None, rows=None):
    g = lib.ssd_logprobs(z, tok.cuda(), K, None if T is None else T.cuda(),
                         rows=None if rows is None else rows.cuda())
    zz = z.cpu() if rows is None else z.cpu()[rows.long()]
    V = zz.shape[1]
    lp, H, rank, top, tlp = ref.logprobs(zz, tok, K, torch.ones(len(tok)) if T is None else T)
    # the sum of V exponentials in 32 bits, at most V / 512 of them one after
    # another, and an argument of at most 2^8 or so rounded twice
    s = (V / 512 + 24) * 2.0 ** -24 + 2.0 ** -20
    _same(g["logprob"], lp, s + lp.abs() * 2.0 ** -21, "logprob")
    _same(g["entropy"], H, s * (2 + 2 * H), "entropy")
    assert torch.equal(g["rank"].cpu().long(), rank.long())
    if K:
        k = min(K, V)
        assert torch.equal(g["top_tok"].cpu().long()[:, :k], top)
        _same(g["top_logprob"][:, :k], tlp, s + tlp.abs() * 2.0 ** -21, "top_logprob")
        assert bool((g["top_tok"][:, k:] == -1).all()) and bool((g["top_logprob"][:, k:] == -math.inf).all())
    assert lib.get_device_error(g["ws"]) == 0
    return g


@pytest.mark.parametrize("R,V,K,dt", [
    (1, 1, 3, torch.float32), (3, 2, 2, BF), (5, 31, 32, torch.float32), (2, 1000, 20, BF), (7, 1001, 5, BF),
    (1, 128256, 5, BF), (40, 4099, 1, torch.float32), (9, 32000, 0, BF), (600, 5000, 8, torch.float32),
    (2, 151936, 32, torch.float32), (3, 151936, 20, BF)])
def test_logprobs(gpu_lib, R, V, K, dt):
    gen = torch.Generator().manual_seed(R + V)
    z = (torch.randn((R, V), generator=gen) * 3).to(dt)
    tok = torch.randint(0, V, (R,), generator=gen).to(torch.int32)
    tok[0] = int(z[0].float().argmax())
    T = torch.rand(R, generator=gen) + 0.4
    _check_logprobs(gpu_lib, z.cuda(), tok, K, T)
    _check_logprobs(gpu_lib, z.cuda(), tok, K)


def test_logprobs_ties_masks_and_order(gpu_lib):
    """Ties go to the lowest index, whatever the order of the values; -inf is a
    masked token; equal rows; rising and falling rows."""
    V = 20000
    z = torch.zeros((8, V))
    z[0, 700:] = 1.0                                     # thousands of equal best
    z[1] = torch.arange(V).float() / 100                 # rising
    z[2] = -torch.arange(V).float() / 100                # falling
    z[3] = -math.inf
    z[3, [5, 19999, 77, 12345]] = torch.tensor([1.0, 2.0, 1.0, 0.0])
    z[4] = -math.inf
    z[4, 123] = -3.0                                     # one token left
    z[5, ::2] = -0.0                                     # -0 and 0 are equal
    z[6] = torch.arange(V).remainder(7).float()
    z[7] = -1e30
    z[7, 9] = 1e30
    tok = torch.tensor([900, 3, 3, 77, 123, 1, 20, 8], dtype=torch.int32)
    for dt in (torch.float32, BF):
        _check_logprobs(gpu_lib, z.to(dt).cuda(), tok, 20)


def test_logprobs_rows_strides_and_unaligned(gpu_lib):
    gen = torch.Generator().manual_seed(5)
    for dt in (torch.float32, BF):
        wide = (torch.randn((6, 3001), generator=gen) * 2).to(dt).cuda()
        rows = torch.tensor([5, 0, 0, 3], dtype=torch.int32)
        tok = torch.tensor([1, 2, 2996, 4], dtype=torch.int32)
        _check_logprobs(gpu_lib, wide[:, 1:2998], tok, 6, rows=rows)
        _check_logprobs(gpu_lib, wide[::2, :2999], tok[:3], 6)


def test_logprobs_refused_rows(gpu_lib):
    z = torch.randn((7, 500), generator=torch.Generator().manual_seed(6))
    z[1, 3], z[2, 499], z[3] = math.nan, math.inf, -math.inf
    rows = torch.tensor([0, 1, 2, 3, -1, 9, 4, 5, 6, 6], dtype=torch.int32)
    tok = torch.tensor([1, 1, 1, 1, 1, 1, 500, -1, 2, 3], dtype=torch.int32)
    T = torch.tensor([1, 1, 1, 1, 1, 1, 1, 1, -1.0, math.nan])
    g = gpu_lib.ssd_logprobs(z.cuda(), tok.cuda(), 3, T.cuda(), rows=rows.cuda())
    lp, H, rk, tt = (g[k].cpu() for k in ("logprob", "entropy", "rank", "top_tok"))
    bad = torch.tensor([0, 1, 1, 1, 1, 1, 0, 0, 1, 1], dtype=torch.bool)
    assert torch.equal(torch.isnan(H), bad) and torch.equal((tt < 0).all(1), bad)
    assert torch.equal(torch.isnan(lp), bad | torch.tensor([0] * 6 + [1, 1, 0, 0], dtype=torch.bool))
    assert rk[0] > 0 and bool((rk[1:] == -1).all())
    E = gpu_lib
    assert E.get_device_error(g["ws"], clear=True) == (
        E.DEVERR_BAD_LOGITS | E.DEVERR_BAD_TEMPERATURE | E.DEVERR_BAD_TOKEN | E.DEVERR_BAD_LENGTH)
    # greedy rows: the one-hot at the lowest argmax
    z = torch.tensor([[1.0, 5.0, 5.0, 2.0]] * 2)
    g = gpu_lib.ssd_logprobs(z.cuda(), torch.tensor([1, 2], dtype=torch.int32).cuda(), 3, torch.zeros(2).cuda())
    assert g["logprob"].tolist() == [0.0, -math.inf] and g["entropy"].tolist() == [0.0, 0.0]
    assert g["rank"].tolist() == [1, 2] and g["top_tok"].tolist() == [[1, 2, 3]] * 2
    assert g["top_logprob"].tolist() == [[0.0, -math.inf, -math.inf]] * 2


def test_operators_graph_capture(gpu_lib):
    """append, commit and logprobs replay from a graph on changed inputs."""
    c = ref.case(2, 4, 4, 2, 64, 16, (20, 30), BF, 40)
    g = ref.to_gpu(c)
    z = torch.randn((4, 3000), device="cuda")
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    acc = torch.ones(2, dtype=torch.int32, device="cuda")
    node = torch.tensor([[3, -1, -1, -1]] * 2, dtype=torch.int32, device="cuda")
    ws = gpu_lib.new_workspace(1 << 20, "cuda")
    o1, o2, o3 = {}, {}, {}

    def step():
        gpu_lib.ssd_kv_append(g["q"], g["k"], g["v"], g["k_cache"], g["v_cache"], g["page_table"],
                              g["ctx_len"], ws=ws, out=o1)
        gpu_lib.ssd_kv_commit(g["k_cache"], g["v_cache"], g["page_table"], g["ctx_len"], acc, node, ws=ws, out=o2)
        gpu_lib.ssd_logprobs(z, tok, 4, ws=ws, out=o3)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g["k"].add_(1)
    z.neg_()
    graph.replay()
    torch.cuda.synchronize()
    for b in range(2):
        L = int(c["ctx_len"][b])
        p, o = ref.where(c, b, L + 1)
        assert torch.equal(g["k_cache"][p, o], g["k"][b, 3])
    assert o2["ctx_len"].tolist() == [22, 32]
    assert torch.equal(o3["top_tok"][:, 0].long(), z.argmax(1))
