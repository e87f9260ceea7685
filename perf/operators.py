"""What the target pass around a verification costs: the operators between the
projections and the logits of a drafted batch, and what a server answers from
the logits.

  append  per-head norms and position rotation of q and k, and k, v stored in
          a paged cache (one layer of a target pass over drafted nodes)
  attn    attention of the drafted nodes (a tree, a chain or one token) over
          the paged cache (one layer)
  commit  the accepted nodes' keys and values moved behind the context, in
          every layer, after the verification
  logp    log probabilities of given tokens, entropy, rank, best alternatives

Head counts, vocabularies, batches and draft lengths are those of the
workloads (B = 1, 64, 512; k = 5, 7; the 21-node tree of widths 4, 2, 1;
V = 128256 and 151936) or generic.  ``own`` selects the library's kernels;
otherwise the operators run in their plain form in float32.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one sequence, a drafted chain of 8 positions, 64 / 8 heads as in a 70B target: latency
        {"name": "attn_b1_chain8", "op": "attn", "B": 1, "N": 8, "Hq": 64, "Hkv": 8, "D": 128, "lo": 4096,
         "hi": 4096, "page": 16, "dtype": "bf16", "tree": "chain", "ragged": False, "order": "slot"},
        # plain decoding of one token a sequence, ragged contexts, small heads, head-major pages
        {"name": "attn_decode_b64_d64", "op": "attn", "B": 64, "N": 1, "Hq": 32, "Hkv": 8, "D": 64, "lo": 200,
         "hi": 6000, "page": 32, "dtype": "f16", "tree": "chain", "ragged": False, "order": "head"},
        # the verification batch: 64 trees of 21 nodes, 168 query rows a KV head, ragged contexts
        {"name": "attn_tree21_b64", "op": "attn", "B": 64, "N": 21, "Hq": 64, "Hkv": 8, "D": 128, "lo": 500,
         "hi": 8000, "page": 16, "dtype": "bf16", "tree": "4,2,1", "ragged": False, "order": "slot"},
        # two long contexts under wide trees of up to 64 nodes
        {"name": "attn_long_tree64", "op": "attn", "B": 2, "N": 64, "Hq": 32, "Hkv": 8, "D": 128, "lo": 60000,
         "hi": 130001, "page": 64, "dtype": "bf16", "tree": "random", "ragged": True, "order": "slot"},
        # one sequence's drafted chain: a launch, little else
        {"name": "append_b1_chain8", "op": "append", "B": 1, "N": 8, "Hq": 64, "Hkv": 8, "D": 128, "lo": 4096,
         "hi": 4096, "page": 16, "dtype": "bf16", "tree": "chain", "ragged": False, "order": "slot", "rot": 128,
         "norm": True, "interleaved": False},
        # the verification batch of trees: packed projections, normed heads
        {"name": "append_tree21_b64", "op": "append", "B": 64, "N": 21, "Hq": 64, "Hkv": 8, "D": 128, "lo": 100,
         "hi": 900, "page": 16, "dtype": "bf16", "tree": "4,2,1", "ragged": False, "order": "slot", "rot": 128,
         "norm": True, "interleaved": False},
        # the large batch of chains: small heads, pairwise rotation of half of each head, no norms
        {"name": "append_b512_d64", "op": "append", "B": 512, "N": 8, "Hq": 32, "Hkv": 8, "D": 64, "lo": 20,
         "hi": 400, "page": 32, "dtype": "f16", "tree": "chain", "ragged": False, "order": "head", "rot": 32,
         "norm": False, "interleaved": True},
        # one accepted path in every layer
        {"name": "commit_b1_l80", "op": "commit", "layers": 80, "B": 1, "N": 21, "Hkv": 8, "D": 128, "lo": 1000,
         "hi": 1000, "page": 16, "dtype": "bf16", "tree": "4,2,1", "order": "slot"},
        # a batch of accepted paths of up to 12 of 64 nodes
        {"name": "commit_b64_l32", "op": "commit", "layers": 32, "B": 64, "N": 64, "Hkv": 8, "D": 128, "lo": 20,
         "hi": 200, "page": 16, "dtype": "bf16", "tree": "random", "order": "slot"},
        # the emitted tokens of one sequence: latency
        {"name": "logp_r8", "op": "logp", "R": 8, "V": 128256, "K": 5, "dtype": "bf16"},
        # the emitted tokens of 64 sequences with the most alternatives an answer carries
        {"name": "logp_r384_k20", "op": "logp", "R": 384, "V": 151936, "K": 20, "dtype": "bf16"},
        # every position of 512 sequences
        {"name": "logp_r4096_f32", "op": "logp", "R": 4096, "V": 151936, "K": 8, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "commit", "logp"])
    if op == "logp":
        V = _log(rng, 1000, 160000)
        return {"op": op, "R": _log(rng, 1, min(4096, 600000000 // V)), "V": V, "K": rng.choice([0, 1, 5, 20, 32]),
                "dtype": rng.choice(["bf16", "f32"])}
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8, 12])
    B = _log(rng, 1, 256)
    N = rng.choice([1, 1, rng.randint(2, 9), rng.randint(10, 40), 64])
    tree = rng.choice(["chain", "random"])
    c = {"op": op, "B": B, "N": N, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "lo": 0, "hi": 0,
         "page": rng.choice([1, 5, 16, 16, 32, 48, 64, 128, 200]), "dtype": rng.choice(["bf16", "f16"]), "tree": tree,
         "ragged": rng.random() < 0.3, "order": rng.choice(["slot", "head"])}
    if op == "attn":
        most = max(16, min(100000, 250000 // B, 60000000 // (B * Hkv * G * N)))
        c["hi"] = _log(rng, 16, most)
        c["lo"] = rng.choice([0, c["hi"] // 10, c["hi"]])
    else:
        c["hi"] = _log(rng, 1, 1000)
        c["lo"] = rng.choice([0, c["hi"]])
    if op == "append":
        c.update(rot=rng.choice([0, 32, D]), norm=rng.random() < 0.5, interleaved=rng.random() < 0.3)
    if op == "commit":
        del c["Hq"], c["ragged"]
        c["layers"] = _log(rng, 1, max(1, min(64, 3000 // B)))
        c["B"] = min(B, 64)
        c["hi"] = min(c["hi"], 300)
        c["lo"] = min(c["lo"], 300)
        c["N"], c["tree"] = max(N, rng.randint(3, 20)), "random"
    return c


# ---------------------------------------------------------------------------
# what a case's numbers mean (no randomness: work() counts the same)
# ---------------------------------------------------------------------------
def _lengths(c):
    """Context lengths from lo to hi, evenly spaced in their logarithm."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    if B == 1:
        return [hi]
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (b / (B - 1)))) - 1 for b in range(B)]


def _node_counts(c):
    return [max(1, c["N"] - b % 3) if c.get("ragged") else c["N"] for b in range(c["B"])]


def _parents(c):
    """[N] parents; -1 at the root."""
    N = c["N"]
    if c["tree"] == "chain":
        return [j - 1 for j in range(N)]
    if c["tree"] == "random":  # breadth-limited: parents a few nodes back
        return [-1] + [max(0, j - 1 - (j * 7 + j * j) % 11) for j in range(1, N)]
    par, level = [-1], [0]
    for w in (int(x) for x in c["tree"].split(",")):
        nxt = []
        for p in level:
            for _ in range(w):
                nxt.append(len(par))
                par.append(p)
        level = nxt
    return par[:N] if len(par) >= N else par + [0] * (N - len(par))


def _paths(c):
    """Accepted path (node ids behind the root) of each sequence: a leaf's
    ancestry cut to a varying depth."""
    par = _parents(c)
    out = []
    for b in range(c["B"]):
        leaf = c["N"] - 1 - (b * 5) % max(1, c["N"] // 2)
        p, j = [], leaf
        while j > 0:
            p.append(j)
            j = par[j]
        p.reverse()
        out.append(p[: max(0, len(p) - b % 3)])
    return out


def work(c):
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "logp":
        n = c["R"] * c["V"]
        return {"bytes": n * e + c["R"] * (20 + 8 * c["K"]), "flops": 6 * n}
    row = c["Hkv"] * c["D"] * e
    if c["op"] == "commit":
        moves = sum(sum(1 for i, j in enumerate(p) if j != i + 1) for p in _paths(c))
        return {"bytes": 4 * c["layers"] * moves * row + c["B"] * (8 + 4 * c["N"]) + 1, "flops": 0}
    nodes = _node_counts(c)
    qrow = c["Hq"] * c["D"] * e
    if c["op"] == "append":
        return {"bytes": sum(nodes) * (2 * (qrow + 2 * row) + 4 * c["rot"]), "flops": sum(nodes) * (qrow + row) * 4}
    pairs = sum(n * (L + n / 2) for n, L in zip(nodes, _lengths(c)))
    return {"bytes": sum(2 * row * (n + L) for n, L in zip(nodes, _lengths(c))) + 2 * c["B"] * c["N"] * qrow,
            "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _cache(c, gen, layers=None):
    """A paged cache with pages in no order, a page table (unused entries -1)
    and the context lengths."""
    B, N, ps, H, D = c["B"], c["N"], c["page"], c["Hkv"], c["D"]
    order = torch.randperm(B, generator=gen, device="cuda").tolist()
    base = _lengths(c)
    lens = [base[i] for i in order]
    need = [-(-(L + N) // ps) for L in lens]
    total, width = sum(need), max(need)
    ids = torch.randperm(total + 3, generator=gen, device="cuda").to(torch.int32)
    # entry (b, p) is page ids[first(b) + p] for p < need(b)
    first = torch.tensor([sum(need[:b]) for b in range(B)] if B < 2 else [0] + torch.tensor(need).cumsum(0)[:-1].tolist(),
                         device="cuda")
    p = torch.arange(width, device="cuda")
    used = p < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(used, ids[(first[:, None] + p).clamp(max=total + 2)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    shape = (total + 3, ps, H, D) if c["order"] == "slot" else (total + 3, H, ps, D)
    if layers is not None:
        shape = (layers,) + shape
    kv = []
    for _ in range(2):
        t = torch.randn(shape, generator=gen, device="cuda", dtype=DTYPES[c["dtype"]])
        kv.append(t if c["order"] == "slot" else t.transpose(-3, -2))
    return {"k_cache": kv[0], "v_cache": kv[1], "page_table": table.contiguous(),
            "ctx_len": torch.tensor(lens, dtype=torch.int32, device="cuda"), "order": order}


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "logp":
        R, V = c["R"], c["V"]
        z = torch.empty((R, V), dtype=dt, device="cuda")
        step = max(1, (1 << 28) // V)
        for r in range(0, R, step):  # N(0, 3) with five peaks, as the verification's logits
            z[r:r + step] = torch.randn((min(step, R - r), V), generator=gen, device="cuda") * 3
        peak = torch.randint(0, V, (R, 5), generator=gen, device="cuda")
        z.scatter_add_(1, peak, torch.full((R, 5), 8.0, dtype=dt, device="cuda"))
        tok = torch.where(torch.rand(R, generator=gen, device="cuda") < 0.7, peak[:, 0],
                          torch.randint(0, V, (R,), generator=gen, device="cuda")).to(torch.int32)
        T = torch.rand(R, generator=gen, device="cuda") * 0.7 + 0.5
        return {"case": c, "logits": z, "tok": tok, "T": T}
    B, N, D = c["B"], c["N"], c["D"]
    s = _cache(c, gen, c.get("layers"))
    s["case"] = c
    order = s.pop("order")
    s["parent"] = torch.tensor(_parents(c), dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    if c["op"] == "commit":
        paths = [_paths(c)[i] for i in order]
        node = torch.full((B, N), -1, dtype=torch.int32)
        for b, p in enumerate(paths):
            node[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        s["out_node"] = node.cuda()
        s["accept_len"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        return s
    nodes = _node_counts(c)
    s["n_nodes"] = torch.tensor([nodes[i] for i in order], dtype=torch.int32, device="cuda") if c["ragged"] else None
    if c["tree"] == "chain":
        s["parent"] = None
    if c["op"] == "attn":
        s["q"] = (torch.randn((B, N, c["Hq"], D), generator=gen, device="cuda") * 2).to(dt)
        return s
    # the projections come packed, one row a token: q heads, k heads, v heads
    packed = torch.randn((B, N, c["Hq"] + 2 * c["Hkv"], D), generator=gen, device="cuda", dtype=dt) * 2
    s["q"], s["k"], s["v"] = packed.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)
    s["cos_sin"] = None
    if c["rot"]:
        f = 500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        ang = torch.arange(c["hi"] + N, dtype=torch.float64, device="cuda")[:, None] * f
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    s["q_norm"] = s["k_norm"] = None
    if c["norm"]:
        s["q_norm"], s["k_norm"] = ((torch.rand(D, generator=gen, device="cuda") + 0.5).to(dt) for _ in range(2))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"attn": _attn, "append": _append, "commit": _commit, "logp": _logp}[s["case"]["op"]](s)


def _run_own(s):
    import speculative_decoding_verification_70_gb300 as ssd
    op = s["case"]["op"]
    out = s.setdefault("out", {})  # outputs and workspace as a decoding loop keeps them
    if op == "attn":
        r = ssd.ssd_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["ctx_len"],
                                   parent=s["parent"], n_nodes=s["n_nodes"], ws=s.get("ws"), out=out)
        s["ws"] = r["ws"]
        return {"out": r["out"], "lse": r["lse"]}
    if op == "append":
        r = ssd.ssd_kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["ctx_len"],
                              parent=s["parent"], n_nodes=s["n_nodes"], cos_sin=s["cos_sin"],
                              interleaved=s["case"]["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6,
                              ws=s.get("ws"), out=out)
        s["ws"] = r["ws"]
        return {"q": r["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "commit":
        r = ssd.ssd_kv_commit(s["k_cache"], s["v_cache"], s["page_table"], s["ctx_len"], s["accept_len"],
                              s["out_node"], ws=s.get("ws"), out=out)
        s["ws"] = r["ws"]
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "ctx_len": r["ctx_len"]}
    r = ssd.ssd_logprobs(s["logits"], s["tok"], s["case"]["K"], s["T"], ws=s.get("ws"), out=out)
    s["ws"] = r["ws"]
    return {k: r[k] for k in ("logprob", "entropy", "rank") + (("top_tok", "top_logprob") if s["case"]["K"] else ())}


def _ancestors(s):
    """[B, N, N] truth values: node i sees node j (its ancestors and itself);
    nodes that a sequence lacks see nothing."""
    c = s["case"]
    B, N = c["B"], c["N"]
    dev = s["ctx_len"].device
    i = torch.arange(N, device=dev)
    if s["parent"] is None:
        see = (i[None, :] <= i[:, None]).expand(B, N, N)
    else:
        up = (s["parent"][:, :, None] == i).float() + torch.eye(N, device=dev)
        see = torch.linalg.matrix_power(up, N) > 0
    if s.get("n_nodes") is not None:
        see = see & (i < s["n_nodes"][:, None])[:, :, None]
    return see


def _attn(s):
    c = s["case"]
    B, N, H, D = c["B"], c["N"], c["Hkv"], c["D"]
    G = c["Hq"] // H
    page = s["page_table"].clamp(min=0).long()
    K, V = (s[n][page].flatten(1, 2).transpose(1, 2).float() for n in ("k_cache", "v_cache"))  # [B, H, S, D]
    S = K.shape[2]
    q = s["q"].float().view(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    see = _ancestors(s)
    node = torch.arange(S, device=q.device) - s["ctx_len"][:, None].long()  # < 0: context
    tree = see.gather(2, node.clamp(0, N - 1)[:, None, :].expand(B, N, S)) & (node < N)[:, None, :]
    there = see.any(2)
    vis = (tree | (node < 0)[:, None, :]) & there[:, :, None]
    vis = vis[:, None, :, None, :].expand(B, H, N, G, S).reshape(B, H, N * G, S)
    x = (q @ K.transpose(2, 3)) * (1.0 / math.sqrt(D))
    x = torch.where(vis, x, torch.full((), -math.inf, device=x.device))
    m = x.amax(3, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp(x - m)
    tot = p.sum(3, keepdim=True)
    V = torch.where((node < N)[:, None, :, None], V, torch.zeros((), device=V.device))
    o = (p @ V) / torch.where(tot > 0, tot, torch.ones_like(tot))
    lse = (m + torch.log(tot))[..., 0]
    o = o.view(B, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, c["Hq"], D)
    lse = lse.view(B, H, N, G).permute(0, 2, 1, 3).reshape(B, N, c["Hq"])
    return {"out": o.to(s["q"].dtype), "lse": lse}


def _rotate(x, cs, sn, interleaved):
    """The first 2 * cs.shape[-1] elements of each head rotated pair by pair."""
    r = cs.shape[-1]
    rot, rest = x[..., :2 * r], x[..., 2 * r:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :r], rot[..., r:])
    u, v = a * cs - b * sn, b * cs + a * sn
    rot = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([rot, rest], -1)


def _append(s):
    c = s["case"]
    N = c["N"]
    see = _ancestors(s)
    there = see.any(2)
    depth = (see.sum(2) - 1).clamp(min=0)
    pos = s["ctx_len"][:, None].long() + depth
    q, k = s["q"].float(), s["k"].float()
    if c["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["q_norm"].float()
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["k_norm"].float()
    if c["rot"]:
        cs, sn = s["cos_sin"][pos].unsqueeze(2).chunk(2, -1)
        q, k = _rotate(q, cs, sn, c["interleaved"]), _rotate(k, cs, sn, c["interleaved"])
    q = torch.where(there[:, :, None, None], q, torch.zeros((), device=q.device))
    slot = s["ctx_len"][:, None].long() + torch.arange(N, device=q.device)
    page = s["page_table"].gather(1, slot // c["page"]).long()
    dst = (page[there], (slot % c["page"])[there])
    s["k_cache"][dst] = k.to(s["k"].dtype)[there]
    s["v_cache"][dst] = s["v"][there]
    return {"q": q.to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _commit(s):
    c = s["case"]
    i = torch.arange(c["N"], device="cuda")
    take = i < s["accept_len"][:, None]
    src = s["ctx_len"][:, None].long() + s["out_node"]
    dst = s["ctx_len"][:, None].long() + 1 + i
    b = torch.arange(c["B"], device="cuda")[:, None].expand_as(take)[take]
    src, dst = src[take], dst[take]
    at = (s["page_table"][b, src // c["page"]].long(), src % c["page"])
    to = (s["page_table"][b, dst // c["page"]].long(), dst % c["page"])
    for t in (s["k_cache"], s["v_cache"]):
        t[:, to[0], to[1]] = t[:, at[0], at[1]]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "ctx_len": s["ctx_len"] + 1 + s["accept_len"]}


def _logp(s):
    z, tok = s["logits"], s["tok"].long()[:, None]
    K, V = s["case"]["K"], z.shape[1]
    T = s["T"][:, None]
    x = z.float() / T
    m = x.amax(1, keepdim=True)
    d = x - m
    w = torch.exp(d)
    tot = w.sum(1, keepdim=True)
    log_tot = torch.log(tot)
    out = {"logprob": (d.gather(1, tok) - log_tot)[:, 0],
           "entropy": (log_tot - (w * d).sum(1, keepdim=True) / tot)[:, 0]}
    del x, d, w
    zf = z.float()
    zt = zf.gather(1, tok)
    idx = torch.arange(V, device=z.device)
    out["rank"] = (1 + ((zf > zt) | ((zf == zt) & (idx < tok))).sum(1)).to(torch.int32)
    if K:
        # one whole-number key orders by value, then by lower index
        bits = (zf + 0.0).view(torch.int32)
        key = (bits ^ ((bits >> 31) & 0x7fffffff)).long() * (1 << 32) + (V - 1 - idx)
        top = (V - 1) - (key.topk(K, 1).values & 0xffffffff)
        out["top_tok"] = top.to(torch.int32)
        out["top_logprob"] = zf.gather(1, top) / T - m - log_tot
    return out


# ---------------------------------------------------------------------------
# the same from the definition, in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------
def _slots(s, b, count):
    """(page, slot) of the first `count` positions of sequence b."""
    n = torch.arange(count, device="cuda")
    ps = s["case"]["page"]
    return s["page_table"][b][n // ps].long(), n % ps


def _seen(par, n):
    """For each of n nodes the list of nodes on its way to the root."""
    out = []
    for j in range(n):
        way, i = [], j
        while i >= 0:
            way.append(i)
            i = par[i]
        out.append(way)
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "logp":
        out = {"logprob": [], "entropy": [], "top_logprob": []}
        for r in range(0, c["R"], 256):
            x = s["logits"][r:r + 256].double() / s["T"][r:r + 256, None].double()
            lp = torch.log_softmax(x, 1)
            out["logprob"].append(lp.gather(1, s["tok"][r:r + 256, None].long())[:, 0])
            out["entropy"].append(-(lp.exp() * lp).sum(1))
            if c["K"]:
                out["top_logprob"].append(lp.topk(c["K"], 1).values)
        out = {k: torch.cat(v) if v else None for k, v in out.items()}
        return {**out, "rank": None, "top_tok": None}
    lens = s["ctx_len"].tolist()
    if c["op"] == "commit":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        for b, L in enumerate(lens):
            path = s["out_node"][b, : int(s["accept_len"][b])].tolist()
            for t, old in ((k, s["k_cache"]), (v, s["v_cache"])):
                for i, j in enumerate(path):
                    (p0, o0), (p1, o1) = (divmod(L + x, c["page"]) for x in (j, i + 1))
                    t[:, int(s["page_table"][b, p1]), o1] = old[:, int(s["page_table"][b, p0]), o0].double()
        return {"k_cache": k, "v_cache": v, "ctx_len": None}
    N, H, D = c["N"], c["Hkv"], c["D"]
    G = c["Hq"] // H
    par = [j - 1 for j in range(N)] if s["parent"] is None else s["parent"][0].tolist()
    counts = [N] * c["B"] if s["n_nodes"] is None else s["n_nodes"].tolist()
    if c["op"] == "attn":
        out = torch.zeros((c["B"], N, c["Hq"], D), dtype=torch.float64, device="cuda")
        lse = torch.full((c["B"], N, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
        for b, L in enumerate(lens):
            n = counts[b]
            page, slot = _slots(s, b, L + n)
            hide = torch.zeros((n, L + n), dtype=torch.bool)
            hide[:, L:] = True
            for i, way in enumerate(_seen(par, n)):
                hide[i, [L + j for j in way]] = False
            hide = hide.cuda()
            for h in range(H):
                K = s["k_cache"][:, :, h][page, slot].double()
                V = s["v_cache"][:, :, h][page, slot].double()
                q = s["q"][b, :n, h * G:(h + 1) * G].double()
                x = torch.einsum("ngd,sd->ngs", q, K) / math.sqrt(D)
                x.masked_fill_(hide[:, None, :], -math.inf)
                lse[b, :n, h * G:(h + 1) * G] = torch.logsumexp(x, 2)
                out[b, :n, h * G:(h + 1) * G] = torch.einsum("ngs,sd->ngd", torch.softmax(x, 2), V)
        return {"out": out, "lse": lse}
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    qo = torch.zeros((c["B"], N, c["Hq"], D), dtype=torch.float64, device="cuda")

    def head(x, w, pos):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
        if c["rot"]:
            r = c["rot"] // 2
            turn = torch.complex(s["cos_sin"][pos, :r].double(), s["cos_sin"][pos, r:].double())[:, None]
            z = x[..., :2 * r]
            z = torch.view_as_complex((z.unflatten(-1, (r, 2)) if c["interleaved"] else z.unflatten(-1, (2, r)).transpose(-1, -2)).contiguous())
            z = torch.view_as_real(z * turn)
            x = torch.cat([(z if c["interleaved"] else z.transpose(-1, -2)).flatten(-2), x[..., 2 * r:]], -1)
        return x

    for b, L in enumerate(lens):
        n = counts[b]
        pos = torch.tensor([L + len(way) - 1 for way in _seen(par, n)], device="cuda")
        page, slot = (t[L:] for t in _slots(s, b, L + n))
        qo[b, :n] = head(s["q"][b, :n], s["q_norm"], pos)
        kc[page, slot] = head(s["k"][b, :n], s["k_norm"], pos)
        vc[page, slot] = s["v"][b, :n].double()
    return {"q": qo, "k_cache": kc, "v_cache": vc}
