"""The example's model with an attention that decides: sharp scores and a large
share of the residual, so that a wrong mask, position or moved slot shows in the
logits.  Against the same decoder in 64 bits without a cache."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import tree_decode as ex  # noqa: E402


def sharp(device):
    """Scores of a deviation of 3, attention eight times the example's."""
    m = ex.Decoder(device=device, seed=4)
    m.q_norm.fill_(3.0)
    for w in m.wo:
        w.mul_(8)
    return m


def exact(m, tok, pos, see, half=lambda t: t):
    """Logits [n, V] of tokens tok [n] at positions pos [n], of which i sees the
    true entries of see[i].  (half: what rounds to 16 bits where the model does)"""
    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def turn(x):  # [n, heads, D], halves apart
        cs, sn = m.cos_sin[pos].double()[:, None].chunk(2, -1)
        a, b = x.chunk(2, -1)
        return torch.cat([a * cs - b * sn, b * cs + a * sn], -1)
    n, G = len(tok), m.Hq // m.Hkv
    x = m.emb[tok].double()
    for i in range(m.layers):
        qkv = half(half(norm(x)) @ m.wqkv[i].double()).view(n, -1, m.D)
        q, k, v = qkv.split([m.Hq, m.Hkv, m.Hkv], 1)
        q = half(turn(norm(q) * m.q_norm.double()))
        k = half(turn(norm(k) * m.k_norm.double())).repeat_interleave(G, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) * m.D ** -0.5
        p = torch.softmax(s.masked_fill(~see, -torch.inf), -1)
        o = half(torch.einsum("hij,jhd->ihd", half(p), v.repeat_interleave(G, 1))).reshape(n, -1)
        x = x + half(o @ m.wo[i].double())
        h = half(torch.nn.functional.silu(half(half(norm(x)) @ m.up[i].double())))
        x = x + half(h @ m.down[i].double())
    return half(half(norm(x)) @ m.head.double())


def layout(ctx, parents):
    """Positions and visible entries of `ctx` committed tokens and a tree behind them."""
    n = ctx + len(parents)
    pos = list(range(ctx))
    see = torch.tril(torch.ones((n, n), dtype=torch.bool))
    for j, p in enumerate(parents):
        see[ctx + j, ctx:] = False
        pos.append(ctx if p < 0 else pos[ctx + p] + 1)
        if p >= 0:
            see[ctx + j] |= see[ctx + p]
        see[ctx + j, ctx + j] = True
    return torch.tensor(pos), see


# The model rounds about ten times a layer to 16 bits, and twice at the end: 22
# errors of about 2^-9 of a vector's length, which add up like independent ones to
# 0.01; those of q and k move scores of a deviation of 3 by 0.02 and weights by 2 %.
# With these roundings emulated on the CPU the logits of 96 nodes are off by 0.012 of
# their length on average and 0.021 at most; sums in another order move either by as
# much again.
TOL = 0.05


def off(got, want):
    return (got.double() - want).norm(dim=-1) / want.norm(dim=-1)


def wrong_masks(ctx, par, see):
    """Masks as mistakes would make them."""
    n = len(par)
    chain = torch.tril(torch.ones_like(see))
    lost, swapped, late = see.clone(), see.clone(), see.clone()
    for j in range(1, n):
        lost[ctx + j, ctx + par[j]] = False                       # the parent is not seen
        twin = next((i for i in range(n) if i != j and par[i] == par[j]), None)
        if twin is not None:
            swapped[ctx + j, ctx + j], swapped[ctx + j, ctx + twin] = False, True  # a sibling's slot for its own
    late[ctx:, ctx - 1] = False                                   # a context one short
    return {"chain": chain, "lost": lost, "swapped": swapped, "late": late}


def test_the_comparison_tells_masks_apart():
    """On the CPU, model and mistakes emulated: the right mask lies well within
    the tolerance, wrong ones well beyond it somewhere."""
    m = sharp("cpu")
    gen = torch.Generator().manual_seed(9)
    ctx, par = 60, ex.tree_parents((3, 2, 1))
    tok = torch.randint(0, m.V, (ctx + len(par),), generator=gen)
    pos, see = layout(ctx, par)
    want = exact(m, tok, pos, see)[ctx:]
    rounded = exact(m, tok, pos, see, lambda t: t.to(torch.bfloat16).double())[ctx:]
    assert float(off(rounded, want).max()) < TOL / 2
    for name, mask in wrong_masks(ctx, par, see).items():
        assert float(off(exact(m, tok, pos, mask)[ctx:], want).max()) > 3 * TOL, name


@pytest.mark.gpu
def test_tree_rounds_against_64_bits(gpu_lib):
    """Three rounds: a prompt, a tree over it, an accepted path that skips nodes,
    the next tree over what was committed.  Every node's logits."""
    m = sharp("cuda")
    gen = torch.Generator().manual_seed(10)
    B, par = 3, ex.tree_parents((3, 2, 1))
    N = len(par)
    parent = torch.tensor(par, dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    prompt = torch.randint(0, m.V, (B, 75), generator=gen)
    cache = ex.PagedCache(m, B, 200)
    ex.prefill(m, cache, prompt[:, :-1].to(torch.int32).cuda())
    done = [prompt[b, :-1].tolist() for b in range(B)]
    paths = [[[3, 8, 14], [2], [1, 5, 11]], [[2, 7], [], [3, 9, 15]], [[1], [3, 8], [2, 6, 12]]]
    for path in paths:
        tok = torch.randint(0, m.V, (B, N), generator=gen)
        got = m.forward(tok.to(torch.int32).cuda(), cache, parent).cpu()
        for b in range(B):
            ctx = len(done[b])
            assert int(cache.ctx_len[b]) == ctx
            pos, see = layout(ctx, par)
            want = exact(m, torch.tensor(done[b] + tok[b].tolist()).cuda(), pos.cuda(), see.cuda())[ctx:].cpu()
            assert float(off(got[b], want).max()) <= TOL
            for i, j in enumerate(path[b]):
                assert par[j] == (path[b][i - 1] if i else 0)
            done[b] += [int(tok[b, 0])] + [int(tok[b, j]) for j in path[b]]
        node = torch.full((B, N), -1, dtype=torch.int32)
        for b in range(B):
            node[b, :len(path[b])] = torch.tensor(path[b], dtype=torch.int32)
        cache.commit(torch.tensor([len(p) for p in path], dtype=torch.int32).cuda(), node.cuda())
    assert not any(cache.errors().values())
