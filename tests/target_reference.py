"""Plain 64-bit forms of the target pass's operators, sequence by sequence,
and seeded inputs for their tests (CPU)."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}  # half a subnormal step


def ways(parent, n):
    """For each node its way to the root (itself first), or None where broken."""
    out = []
    for j in range(n):
        way, i = [j], j
        while i > 0:
            p = parent[i]
            if p < 0 or p >= i:
                way = None
                break
            way.append(p)
            i = p
        out.append(way if way is not None and (parent[0] == -1) else None)
    return out


def nodes_of(c, b):
    """(n, ways) of sequence b: n = 0 where its lengths are out of range."""
    N = c["N"]
    n = N if c.get("n_nodes") is None else int(c["n_nodes"][b])
    L = int(c["ctx_len"][b])
    room = c["page_table"].shape[1] * c["page"]
    if L < 0 or n < 0 or n > N or L + n > room:
        return 0, []
    par = list(range(-1, N - 1)) if c.get("parent") is None else c["parent"][b].tolist()
    return n, ways(par, n)


def where(c, b, slot):
    """(page, entry) of a slot, page -1 for one that the cache does not hold."""
    page = int(c["page_table"][b, slot // c["page"]])
    return (page if 0 <= page < c["k_cache"].shape[0] else -1), slot % c["page"]


def gather(c, b, slots, cache):
    """[len, H, D] in 64 bits; zeros for a bad page."""
    rows = []
    for s in slots:
        p, o = where(c, b, s)
        rows.append(cache[p, o].double() if p >= 0 else torch.zeros(cache.shape[2:], dtype=torch.float64))
    return torch.stack(rows)


def attention(c, scale=None):
    """out, lse and the tolerance of each out entry and lse (in 64 bits)."""
    q = c["q"]
    B, N, Hq, D = q.shape
    H = c["k_cache"].shape[2]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    half, tiny = HALF_STEP[q.dtype], TINY[q.dtype]
    for b in range(B):
        n, way = nodes_of(c, b)
        L = int(c["ctx_len"][b])
        if n == 0 or all(w is None for w in way):
            continue
        K = gather(c, b, range(L + n), c["k_cache"])
        V = gather(c, b, range(L + n), c["v_cache"])
        for i in range(n):
            if way[i] is None:
                continue
            seen = list(range(L)) + sorted(L + j for j in way[i])
            k, v = K[seen].repeat_interleave(G, 1), V[seen].repeat_interleave(G, 1)  # [S, Hq, D]
            qi = q[b, i].double()
            x = torch.einsum("hd,shd->hs", qi, k) * scale
            p = torch.softmax(x, 1)
            o = torch.einsum("hs,shd->hd", p, v)
            out[b, i], lse[b, i] = o, torch.logsumexp(x, 1)
            # a score is a sum of D products in 32 bits; p is rounded to 16 bits
            # before its product with v, the result once more
            d = (D + 4) * 2.0 ** -24 * torch.einsum("hd,shd->hs", qi.abs(), k.abs()).amax(1) * abs(scale)
            w = torch.einsum("hs,shd->hd", p, v.abs())
            fp16 = len(seen) * tiny * v.abs().amax(0)
            tol[b, i] = half * o.abs() + w * (half + 2 * d[:, None] + 2.0 ** -18) + fp16 + tiny
            ltol[b, i] = d + 2.0 ** -18 + lse[b, i].abs() * 2.0 ** -22
    return out, lse, tol, ltol


def append(c, rot=0, interleaved=False, eps=1e-6):
    """q_out, k_cache, v_cache after the append, and tolerances of q_out and
    k_cache."""
    q, k, v = c["q"], c["k"], c["v"]
    kc, vc = c["k_cache"].double(), c["v_cache"].double()
    qo = torch.zeros(q.shape, dtype=torch.float64)
    qt, kt = torch.zeros_like(qo), torch.zeros_like(kc)
    half, tiny = HALF_STEP[q.dtype], TINY[q.dtype]

    def head(x, w, pos):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
        y, size = x.clone(), x.abs()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            cs, sn = float(c["cos_sin"][pos, i]), float(c["cos_sin"][pos, i + rot // 2])
            y[..., a] = x[..., a] * cs - x[..., b] * sn
            y[..., b] = x[..., b] * cs + x[..., a] * sn
            size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
        # one rounding to 16 bits; in 32 bits a sum of D squares, a root, a
        # quotient and five products or sums
        return y, half * y.abs() + 2.0 ** -19 * size + tiny

    for b in range(q.shape[0]):
        n, way = nodes_of(c, b)
        L = int(c["ctx_len"][b])
        for j in range(n):
            if way[j] is None:
                continue
            pos = L + len(way[j]) - 1
            if rot and pos >= c["cos_sin"].shape[0]:
                continue
            qo[b, j], qt[b, j] = head(q[b, j], c.get("q_norm"), pos)
            p, o = where(c, b, L + j)
            if p >= 0:
                kc[p, o], kt[p, o] = head(k[b, j], c.get("k_norm"), pos)
                vc[p, o] = v[b, j].double()
    if rot == 0 and c.get("q_norm") is None:
        qt.zero_(), kt.zero_()  # copies
    return qo, kc, vc, qt, kt


def logprobs(z, tok, K, T):
    """Per answer: logprob, entropy, rank, top tokens and their logprobs, of
    rows z [R, V] (valid rows, T > 0)."""
    x = z.double() / T.double()[:, None]
    lp = torch.log_softmax(x, 1)
    p = lp.exp()
    H = -(torch.where(p > 0, p * lp, torch.zeros_like(p))).sum(1)
    order = torch.sort(z.double(), dim=1, descending=True, stable=True).indices
    rank = (order == tok[:, None]).int().argmax(1) + 1
    top = order[:, :K]
    return lp.gather(1, tok[:, None].long())[:, 0], H, rank, top, lp.gather(1, top)


def random_tree(N, gen, chainish=0.5):
    par = [-1]
    for j in range(1, N):
        if float(torch.rand((), generator=gen)) < chainish:
            par.append(j - 1)
        else:
            par.append(int(torch.randint(0, j, (), generator=gen)))
    return par


def case(B, N, Hq, Hkv, D, page, ctx, dtype, seed, tree="random", ragged=False, order="slot",
         fill="random", spare=2, width_extra=0, packed=False):
    """Seeded inputs on the CPU.  fill="nan": every slot that no node sees
    holds NaN."""
    g = torch.Generator().manual_seed(seed)
    ctx = list(ctx) if not isinstance(ctx, int) else [ctx] * B
    need = [max(1, -(-(L + N) // page)) for L in ctx]
    width = max(need) + width_extra
    pages = sum(need) + spare
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    shape = (pages, page, Hkv, D) if order == "slot" else (pages, Hkv, page, D)
    kv = [torch.randn(shape, generator=g).to(dtype) for _ in range(2)]
    if order == "head":
        kv = [t.transpose(1, 2) for t in kv]
    c = {"N": N, "page": page, "ctx_len": torch.tensor(ctx, dtype=torch.int32), "page_table": table,
         "k_cache": kv[0], "v_cache": kv[1], "parent": None, "n_nodes": None}
    if tree == "random":
        c["parent"] = torch.tensor([random_tree(N, g) for _ in range(B)], dtype=torch.int32)
    if ragged:
        c["n_nodes"] = torch.tensor([(b * 7) % (N + 1) for b in range(B)], dtype=torch.int32)
    if packed:
        x = torch.randn((B, N, Hq + 2 * Hkv, D), generator=g).to(dtype) * 2
        c["q"], c["k"], c["v"] = x.split([Hq, Hkv, Hkv], 2)
    else:
        c["q"] = (torch.randn((B, N, Hq, D), generator=g) * 2).to(dtype)
        c["k"], c["v"] = (torch.randn((B, N, Hkv, D), generator=g).to(dtype) for _ in range(2))
    if fill == "nan":
        keep = torch.zeros((pages, page), dtype=torch.bool)
        for b in range(B):
            n, _ = nodes_of(c, b)
            for s in range(ctx[b] + n):
                p, o = where(c, b, s)
                keep[p, o] = True
        for t in kv:
            t[~keep] = math.nan
    return c


def to_gpu(c):
    """The same on the GPU, strides kept."""
    out = {}
    for k, v in c.items():
        if isinstance(v, torch.Tensor):
            if v.dim() == 4 and not v.is_contiguous() and v.transpose(1, 2).is_contiguous():
                v = v.transpose(1, 2).cuda().transpose(1, 2)
            else:
                v = v.cuda()
        out[k] = v
    if isinstance(c.get("q"), torch.Tensor) and not c["q"].is_contiguous():  # packed projection
        x = torch.cat([c["q"], c["k"], c["v"]], 2).cuda()
        H = c["k"].shape[2]
        out["q"], out["k"], out["v"] = x.split([c["q"].shape[2], H, H], 2)
    return out
