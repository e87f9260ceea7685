"""Plain 64-bit forms of the operators of prompts and budgets (chunk attention, summed
weights, eviction), sequence by sequence, and their tolerances (CPU)."""
import math

import torch

import target_reference as ref

HALF_STEP, TINY = ref.HALF_STEP, ref.TINY


def tokens_of(c, b):
    """New tokens of sequence b: 0 where its lengths are out of range."""
    return ref.nodes_of(c, b)[0] if c["N"] <= 64 else _count(c, b)


def _count(c, b):
    n = c["N"] if c.get("n_nodes") is None else int(c["n_nodes"][b])
    L = int(c["ctx_len"][b])
    return 0 if L < 0 or n < 0 or n > c["N"] or L + n > c["page_table"].shape[1] * c["page"] else n


def gather(c, b, count, cache):
    """[count, H, D] in 64 bits; zeros for a bad page."""
    ps = c["page"]
    s = torch.arange(count)
    page = c["page_table"][b][s // ps].long()
    good = (page >= 0) & (page < cache.shape[0])
    x = cache[page.clamp(0, cache.shape[0] - 1), s % ps].double()
    x[~good] = 0
    return x


def seen(L, n, window, sinks):
    """[n, L + n] truth values: which slots the new tokens see."""
    p = L + torch.arange(n)[:, None]
    s = torch.arange(L + n)[None, :]
    m = s <= p
    if window:
        m = m & ((s > p - window) | (s < sinks))
    return m


def attention(c, window=0, sinks=0, scale=None):
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
        n, L = tokens_of(c, b), int(c["ctx_len"][b])
        if n == 0:
            continue
        K, V = gather(c, b, L + n, c["k_cache"]), gather(c, b, L + n, c["v_cache"])
        see = seen(L, n, window, sinks)
        bad = ~torch.isfinite(V).all(2).all(1)  # slots with NaN or infinite values
        for h in range(H):
            qh = q[b, :n, h * G:(h + 1) * G].double()
            x = torch.einsum("ngd,sd->ngs", qh, K[:, h]) * scale
            x = torch.where(see[:, None, :], x, torch.full((), -math.inf, dtype=torch.float64))
            m = x.amax(2, keepdim=True)
            p = torch.where(see[:, None, :], torch.exp(x - torch.where(m > -math.inf, m, 0 * m)), 0 * m)
            l = p.sum(2, keepdim=True)
            p = p / torch.where(l == 0, torch.ones_like(l), l)
            fine = torch.where(bad[:, None], 0 * V[:, h], V[:, h])
            fine = torch.where(torch.isfinite(fine), fine, torch.zeros_like(fine))
            o = torch.einsum("ngs,sd->ngd", p, fine)
            for s in bad.nonzero()[:, 0].tolist():
                rows = see[:, s]
                o[rows] += p[rows][:, :, s, None] * V[s, h]
            # a score is a sum of D products in 32 bits; p is rounded to 16 bits before its
            # product with v, the result once more
            size = torch.einsum("ngd,sd->ngs", qh.abs(), K[:, h].abs().nan_to_num(0, 0, 0))
            d = (D + 4) * 2.0 ** -24 * torch.where(see[:, None, :], size, 0 * size).amax(2) * abs(scale)
            # (finite entries of slots that hold others count like all)
            fine = torch.where(torch.isfinite(V[:, h]), V[:, h], torch.zeros_like(V[:, h]))
            w = torch.einsum("ngs,sd->ngd", p.nan_to_num(0), fine.abs())
            far = torch.where(see[:, None, :], x, 0 * x).abs().nan_to_num(0, 0, 0).amax(2)
            d = d + far * 2.0 ** -23  # the scaled score, and its distance from the reference
            fp16 = see.sum(1)[:, None, None] * tiny * fine.abs().amax(0)
            at = slice(h * G, (h + 1) * G)
            out[b, :n, at] = o
            lse[b, :n, at] = m[..., 0] + torch.log(l[..., 0])
            tol[b, :n, at] = half * o.abs() + w * (half + 2 * d[..., None] + 2.0 ** -18) + fp16 + tiny
            ltol[b, :n, at] = d + 2.0 ** -18 + lse[b, :n, at].abs() * 2.0 ** -22
    return out, lse, tol, ltol


def weights(c, lse, w, window=0, sinks=0, scale=None, decay=1.0):
    """w [B, Hkv, S] afterwards and its tolerance; lse [B, N, Hq] as the call gets it."""
    q = c["q"]
    B, N, Hq, D = q.shape
    H = c["k_cache"].shape[2]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out, tol = w.double().clone(), torch.zeros(w.shape, dtype=torch.float64)
    for b in range(B):
        n, L = tokens_of(c, b), int(c["ctx_len"][b])
        if n == 0 or L + n > w.shape[2]:
            continue
        K = gather(c, b, L + n, c["k_cache"])
        see = seen(L, n, window, sinks)[:, None, :]
        for h in range(H):
            qh = q[b, :n, h * G:(h + 1) * G].double()
            x = torch.einsum("ngd,sd->ngs", qh, K[:, h]) * scale
            y = lse[b, :n, h * G:(h + 1) * G, None].double()
            p = torch.where(see & (y > -math.inf), torch.exp(x - y), torch.zeros_like(x))
            old = 0 if decay == 0 else w[b, h, :L + n].double() * decay
            out[b, h, :L + n] = old + p.sum((0, 1))
            # scores as above; the exponential two units of the last place, its argument rounded
            # at the size of the score and of lse; sums of non-negative terms in 32 bits
            size = torch.einsum("ngd,sd->ngs", qh.abs(), K[:, h].abs().nan_to_num(0, 0, 0))
            d = (D + 4) * 2.0 ** -24 * size * abs(scale) + (x.abs() + y.abs()).nan_to_num(0, 0, 0) * 2.0 ** -22
            terms = 2 * n * G
            tol[b, h, :L + n] = (p.nan_to_num(0) * (d + 2.0 ** -21)).sum((0, 1)) + terms * 2.0 ** -24 * out[
                b, h, :L + n].abs().nan_to_num(0, 0, 0) + n * G * 2.0 ** -126
    return out, tol


def order_of(w):
    """Slots of one row, heaviest first: equal ones by slot, -0 as 0, NaN last."""
    v = [(-math.inf if x != x else x, x == x, -s) for s, x in enumerate(w.tolist())]
    return sorted(range(len(v)), key=lambda s: (v[s][1], v[s][0], v[s][2]), reverse=True)


def evict(c, w, budget, sinks=0, recent=0):
    """k_cache, v_cache, ctx_len, kept, weights afterwards; caches [layers, ...] and w
    [layers, B, H, S] on the CPU."""
    k, v = c["k_cache"].clone(), c["v_cache"].clone()
    layers, B, H, S = w.shape
    new = c["ctx_len"].clone()
    kept = torch.full((layers, B, H, budget), -1, dtype=torch.int32)
    wout = torch.zeros_like(w)
    ps, pages = c["page"], k.shape[1]
    for b in range(B):
        L = int(c["ctx_len"][b])
        if L < 0 or L > S or L > c["page_table"].shape[1] * ps:
            wout[:, b] = math.nan  # not written
            continue
        new[b] = min(L, budget)
        for layer in range(layers):
            for h in range(H):
                if L <= budget:
                    keep = list(range(L))
                else:
                    mid = order_of(w[layer, b, h, sinks:L - recent])[:budget - sinks - recent]
                    keep = list(range(sinks)) + sorted(sinks + s for s in mid) + list(range(L - recent, L))
                kept[layer, b, h, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
                wout[layer, b, h, :len(keep)] = w[layer, b, h, torch.tensor(keep, dtype=torch.long)]
                if L <= budget:
                    continue
                for r, s in enumerate(keep):
                    p0, p1 = int(c["page_table"][b, s // ps]), int(c["page_table"][b, r // ps])
                    if 0 <= p0 < pages and 0 <= p1 < pages:
                        k[layer, p1, r % ps, h] = c["k_cache"][layer, p0, s % ps, h]
                        v[layer, p1, r % ps, h] = c["v_cache"][layer, p0, s % ps, h]
    return k, v, new, kept, wout
