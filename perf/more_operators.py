"""What prompts and budgets cost over a paged cache: the operators that fill a
cache with prompts, look at a part of it, and cut it down.

  attn   attention of chunks of new tokens (prompts, drafted chains, single
         tokens) over the cache, causal, with or without a sliding window and
         first tokens that stay visible (one layer)
  sum    attention weights of the same tokens added up for every slot (one layer)
  evict  the heaviest slots kept within a budget, every head by its own weights,
         and moved to the front of the cache (all layers)

Head counts, batches, draft lengths, page sizes and contexts are those of the
workloads and of the paged cache's tests, or generic.  ``own`` selects the
library's kernels; otherwise the operators run in their plain form in float32.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a drafted chain of 8 positions behind a long context of which a window is seen: latency
        {"name": "attn_b1_chain8_window", "op": "attn", "B": 1, "N": 8, "Hq": 64, "Hkv": 8, "D": 128, "lo": 131000,
         "hi": 131000, "page": 16, "dtype": "bf16", "ragged": False, "order": "slot", "window": 4096, "sinks": 4},
        # plain decoding of one token a sequence under a window, ragged contexts, small heads, head-major pages
        {"name": "attn_decode_b64_window", "op": "attn", "B": 64, "N": 1, "Hq": 32, "Hkv": 8, "D": 64, "lo": 200,
         "hi": 20000, "page": 32, "dtype": "f16", "ragged": False, "order": "head", "window": 2048, "sinks": 16},
        # a batch of chunks of all lengths under a window, five query heads a group, odd sizes
        {"name": "attn_ragged_b12_window", "op": "attn", "B": 12, "N": 1501, "Hq": 40, "Hkv": 8, "D": 64, "lo": 0,
         "hi": 6000, "page": 48, "dtype": "f16", "ragged": True, "order": "slot", "window": 1000, "sinks": 130},
        # a whole prompt, 64 / 8 heads as in a 70B target
        {"name": "attn_prompt_8k", "op": "attn", "B": 1, "N": 8192, "Hq": 64, "Hkv": 8, "D": 128, "lo": 0, "hi": 0,
         "page": 16, "dtype": "bf16", "ragged": False, "order": "slot", "window": 0, "sinks": 0},
        # a chunk of a long prompt
        {"name": "attn_chunk2k_at60k", "op": "attn", "B": 1, "N": 2048, "Hq": 32, "Hkv": 8, "D": 128, "lo": 60001,
         "hi": 60001, "page": 64, "dtype": "bf16", "ragged": False, "order": "slot", "window": 0, "sinks": 0},
        # the weights of one token a sequence, added to those of the steps before
        {"name": "sum_decode_b64", "op": "sum", "B": 64, "N": 1, "Hq": 64, "Hkv": 8, "D": 128, "lo": 200, "hi": 8000,
         "page": 16, "dtype": "bf16", "ragged": False, "order": "slot", "window": 0, "sinks": 0, "decay": 1.0},
        # the last 32 tokens of a long prompt as observers, into new weights
        {"name": "sum_b1_observe32", "op": "sum", "B": 1, "N": 32, "Hq": 32, "Hkv": 8, "D": 128, "lo": 60001,
         "hi": 60001, "page": 16, "dtype": "bf16", "ragged": False, "order": "slot", "window": 0, "sinks": 0,
         "decay": 0.0},
        # whole prompts as observers, older weights fading
        {"name": "sum_prompts_b4", "op": "sum", "B": 4, "N": 2500, "Hq": 32, "Hkv": 8, "D": 64, "lo": 0, "hi": 3000,
         "page": 32, "dtype": "f16", "ragged": True, "order": "head", "window": 0, "sinks": 0, "decay": 0.9},
        # one sequence cut to its budget, 80 layers
        {"name": "evict_b1_l80", "op": "evict", "layers": 80, "B": 1, "Hkv": 8, "D": 128, "lo": 4096, "hi": 4096,
         "page": 16, "dtype": "bf16", "order": "slot", "budget": 1024, "sinks": 4, "recent": 256},
        # one long sequence cut far down, few layers
        {"name": "evict_b1_100k", "op": "evict", "layers": 2, "B": 1, "Hkv": 8, "D": 128, "lo": 100003, "hi": 100003,
         "page": 64, "dtype": "bf16", "order": "slot", "budget": 8192, "sinks": 16, "recent": 1024},
        # a batch of ragged contexts, some within the budget
        {"name": "evict_b64_l4", "op": "evict", "layers": 4, "B": 64, "Hkv": 8, "D": 64, "lo": 500, "hi": 9001,
         "page": 32, "dtype": "f16", "order": "head", "budget": 1500, "sinks": 4, "recent": 500},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "sum", "evict"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    c = {"op": op, "Hkv": Hkv, "D": D, "page": rng.choice([1, 5, 16, 16, 32, 48, 64, 128, 200]),
         "dtype": rng.choice(["bf16", "f16"]), "order": rng.choice(["slot", "head"])}
    if op == "evict":
        B = _log(rng, 1, 64)
        layers = _log(rng, 1, max(1, min(80, 256 // B)))
        hi = _log(rng, 8, min(100000, 6000000 // (B * layers)))
        budget = max(1, int(hi * rng.uniform(0.05, 1.1)))
        sinks = rng.choice([0, min(4, budget // 4), budget // 3])
        recent = rng.choice([0, budget // 4, budget // 2])
        return {**c, "B": B, "layers": layers, "lo": rng.choice([0, hi // 3, hi]), "hi": hi, "budget": budget,
                "sinks": sinks, "recent": recent}
    G = rng.choice([1, 2, 4, 5, 7, 8, 12])
    B = _log(rng, 1, 64)
    N = rng.choice([1, rng.randint(2, 30), _log(rng, 30, max(31, min(4000, 16000 // B)))])
    # as many scores as the plain form holds at once
    hi = _log(rng, 16, max(32, min(100000, 400000 // B, 1500000000 // (B * Hkv * G * N))))
    return {**c, "B": B, "N": N, "Hq": Hkv * G, "lo": rng.choice([0, hi // 10, hi]), "hi": hi,
            "ragged": rng.random() < 0.4, "window": rng.choice([0, 0, 17, 128, 1000, 4096]),
            "sinks": rng.choice([0, 1, 4, 64, 130]), **({"decay": rng.choice([0.0, 0.9, 1.0])} if op == "sum" else {})}


# ---------------------------------------------------------------------------
# what a case's numbers mean (no randomness: work() counts the same)
# ---------------------------------------------------------------------------
def _lengths(c):
    """Context lengths from lo to hi, evenly spaced in their logarithm."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    if B == 1:
        return [hi]
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (b / (B - 1)))) - 1 for b in range(B)]


def _new_tokens(c):
    """New tokens of each sequence: N, or eighths of it and none for every seventh."""
    if not c.get("ragged"):
        return [c["N"]] * c["B"]
    return [0 if b % 7 == 6 else max(1, c["N"] * ((b * 5 + 7) % 8 + 1) // 8) for b in range(c["B"])]


def _seen(c, ctx, n):
    """(slots that some token sees, sum over the tokens of the slots each sees)."""
    W, K = c["window"], c["sinks"]
    if n == 0:
        return 0, 0
    if W == 0:
        return ctx + n, n * ctx + n * (n + 1) // 2
    pairs = 0
    for p in range(ctx, ctx + n):
        first = max(0, p + 1 - W)
        pairs += p + 1 - first + min(K, first)
    first = max(0, ctx + 1 - W)
    return ctx + n - first + min(K, first), pairs


def work(c):
    row = c["Hkv"] * c["D"] * 2
    if c["op"] == "evict":
        heads = c["layers"] * c["Hkv"]
        slots = sum(_lengths(c))
        moved = sum(c["budget"] - c["sinks"] for L in _lengths(c) if L > c["budget"])
        return {"bytes": heads * 4 * (slots + c["B"] * (c["budget"] + c["hi"])) + 4 * c["layers"] * moved * row,
                "flops": 0}
    seen = [_seen(c, L, n) for L, n in zip(_lengths(c), _new_tokens(c))]
    slots, pairs = sum(s for s, _ in seen), sum(p for _, p in seen)
    q = sum(_new_tokens(c)) * c["Hq"]
    if c["op"] == "attn":
        return {"bytes": 2 * row * slots + q * (4 * c["D"] + 4), "flops": 4 * pairs * c["Hq"] * c["D"]}
    every = sum(L + n for L, n in zip(_lengths(c), _new_tokens(c)) if n)
    return {"bytes": row * slots + q * (2 * c["D"] + 4) + c["Hkv"] * (4 if c["decay"] == 0 else 8) * every,
            "flops": 2 * pairs * c["Hq"] * c["D"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _cache(c, gen, extra, layers=None):
    """A paged cache with pages in no order, a page table (unused entries -1)
    and the context lengths, of the sequences in no order."""
    B, ps, H, D = c["B"], c["page"], c["Hkv"], c["D"]
    order = torch.randperm(B, generator=gen, device="cuda").tolist()
    base, more = _lengths(c), extra
    lens = [base[i] for i in order]
    need = [max(1, -(-(base[i] + more[i]) // ps)) for i in order]
    total, width = sum(need), max(need)
    ids = torch.randperm(total + 3, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor([0] + torch.tensor(need).cumsum(0)[:-1].tolist(), device="cuda")
    p = torch.arange(width, device="cuda")
    used = p < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(used, ids[(first[:, None] + p).clamp(max=total + 2)],
                        torch.full((), -1, dtype=torch.int32, device="cuda"))
    shape = (total + 3, ps, H, D) if c["order"] == "slot" else (total + 3, H, ps, D)
    if layers is not None:
        shape = (layers,) + shape
    kv = []
    for _ in range(2):
        t = torch.randn(shape, generator=gen, device="cuda", dtype=DTYPES[c["dtype"]])
        kv.append(t if c["order"] == "slot" else t.transpose(-3, -2))
    return {"k_cache": kv[0], "v_cache": kv[1], "page_table": table.contiguous(),
            "ctx_len": torch.tensor(lens, dtype=torch.int32, device="cuda")}, order


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if c["op"] == "evict":
        s, _ = _cache(c, gen, [0] * c["B"], c["layers"])
        # weights as a cache collects them: few heavy slots, many light ones, some never
        # looked at, and enough equal ones for ties
        w = torch.exp(torch.randn((c["layers"], c["B"], c["Hkv"], max(1, c["hi"])), generator=gen, device="cuda") * 2)
        w = w.to(torch.bfloat16).float()
        s["weights"] = torch.where(w < 0.15, torch.zeros_like(w), w)
        s["case"] = c
        return s
    N = c["N"]
    new = _new_tokens(c)
    s, order = _cache(c, gen, new)
    s["case"] = c
    s["n_nodes"] = torch.tensor([new[i] for i in order], dtype=torch.int32, device="cuda") if c["ragged"] else None
    s["q"] = (torch.randn((c["B"], N, c["Hq"], c["D"]), generator=gen, device="cuda") * 2).to(DTYPES[c["dtype"]])
    if c["op"] == "sum":
        x = _scores(s)
        s["lse"] = _to_tokens(s, torch.logsumexp(x, 3)[..., None])[..., 0].contiguous()
        del x
        s["weights"] = torch.rand((c["B"], c["Hkv"], c["hi"] + N), generator=gen, device="cuda") * 3
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"attn": _attn, "sum": _sum, "evict": _evict}[s["case"]["op"]](s)


def _run_own(s):
    import speculative_decoding_verification_70_gb300 as ssd
    c = s["case"]
    out = s.setdefault("out", {})  # outputs and workspace as a decoding loop keeps them
    if c["op"] == "attn":
        r = ssd.ssd_chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["ctx_len"],
                                    n_nodes=s["n_nodes"], window=c["window"], sinks=c["sinks"], ws=s.get("ws"), out=out)
        s["ws"] = r["ws"]
        return {"out": r["out"], "lse": r["lse"]}
    if c["op"] == "sum":
        r = ssd.ssd_kv_weights(s["q"], s["k_cache"], s["page_table"], s["ctx_len"], s["lse"], s["weights"],
                               n_nodes=s["n_nodes"], window=c["window"], sinks=c["sinks"], decay=c["decay"],
                               ws=s.get("ws"))
        s["ws"] = r["ws"]
        return {"weights": r["weights"]}
    r = ssd.ssd_kv_evict(s["k_cache"], s["v_cache"], s["page_table"], s["ctx_len"], s["weights"], c["budget"],
                         sinks=c["sinks"], recent=c["recent"], ws=s.get("ws"), out=out)
    s["ws"] = r["ws"]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "ctx_len": r["ctx_len"], "kept": r["kept"],
            "weights": r["weights"]}


def _visible(s, S):
    """([B, N, S] truth values, which token sees which slot; [B, N], which tokens are there)."""
    c = s["case"]
    i, slot = torch.arange(c["N"], device="cuda"), torch.arange(S, device="cuda")
    n = s["n_nodes"] if s["n_nodes"] is not None else torch.full_like(s["ctx_len"], c["N"])
    there = i < n[:, None]
    pos = (s["ctx_len"][:, None] + i)[:, :, None]
    see = slot <= pos
    if c["window"]:
        see &= (slot > pos - c["window"]) | (slot < c["sinks"])
    return see & there[:, :, None], there


def _rows(s, cache):
    """[B, Hkv, S, D] in float32: every sequence's slots in order."""
    return cache[s["page_table"].clamp(min=0).long()].flatten(1, 2).transpose(1, 2).float()


def _scores(s):
    """[B, Hkv, N * G, S] in float32, -inf where a token does not see a slot."""
    c = s["case"]
    B, N, H, D = c["B"], c["N"], c["Hkv"], c["D"]
    G = c["Hq"] // H
    K = _rows(s, s["k_cache"])
    q = s["q"].float().view(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    x = (q @ K.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, H, N, G, -1)
    see, _ = _visible(s, K.shape[2])
    return x.masked_fill_(~see[:, None, :, None, :], -math.inf).flatten(2, 3)


def _to_tokens(s, o):
    """[B, N, Hq, ...] of [B, Hkv, N * G, ...]."""
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    return o.view(c["B"], c["Hkv"], c["N"], G, -1).permute(0, 2, 1, 3, 4).reshape(c["B"], c["N"], c["Hq"], -1)


def _attn(s):
    x = _scores(s)
    m = x.amax(3, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = x.sub_(m).exp_()
    tot = p.sum(3, keepdim=True)
    # slots behind a sequence's end hold nothing
    n = s["n_nodes"] if s["n_nodes"] is not None else s["case"]["N"]
    end = (s["ctx_len"] + n)[:, None, None, None]
    V = _rows(s, s["v_cache"])
    V = torch.where(torch.arange(V.shape[2], device="cuda")[:, None] < end, V, torch.zeros((), device="cuda"))
    o = (p @ V) / torch.where(tot > 0, tot, torch.ones_like(tot))
    return {"out": _to_tokens(s, o).to(s["q"].dtype), "lse": _to_tokens(s, m + torch.log(tot))[..., 0].contiguous()}


def _sum(s):
    c = s["case"]
    x = _scores(s)
    G = c["Hq"] // c["Hkv"]
    lse = s["lse"].view(c["B"], c["N"], c["Hkv"], G).permute(0, 2, 1, 3).reshape(c["B"], c["Hkv"], -1, 1)
    lse = torch.where(lse > -math.inf, lse, torch.zeros_like(lse))
    w = x.sub_(lse).exp_().sum(2)
    W = s["weights"]
    n = s["n_nodes"] if s["n_nodes"] is not None else torch.full_like(s["ctx_len"], c["N"])
    end = torch.where(n > 0, s["ctx_len"] + n, torch.zeros_like(n))
    S = min(W.shape[2], w.shape[2])
    touched = (torch.arange(S, device="cuda") < end[:, None])[:, None, :]
    W[:, :, :S] = torch.where(touched, W[:, :, :S] * c["decay"] + w[:, :, :S], W[:, :, :S])
    return {"weights": W}


def _evict(s):
    c = s["case"]
    L, B, H, S = s["weights"].shape
    C = c["budget"]
    ctx = s["ctx_len"].long()[:, None, None]
    slot = torch.arange(S, device="cuda")
    bits = (s["weights"] + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7fffffff)).long()  # ordered as the weights are
    key = torch.where((slot < c["sinks"]) | (slot >= ctx - c["recent"]), 1 << 31, key)
    key = torch.where(slot < ctx, key, -(1 << 31) - 1)
    key = key * (1 << 30) + (S - 1 - slot)             # equal weights: the lower slot first
    k = min(C, S)
    kept = (S - 1 - (key.topk(k, 3).values & ((1 << 30) - 1)))
    kept = torch.where(kept < ctx, kept, S).sort(3).values
    new_len = s["ctx_len"].clamp(max=C)
    there = torch.arange(k, device="cuda") < new_len[:, None, None].long()
    there = there.expand(L, B, H, k)
    kept = torch.where(there, kept, torch.full_like(kept, -1))
    src = kept.clamp(min=0)
    wout = torch.zeros_like(s["weights"])
    wout[..., :k] = torch.where(there, s["weights"].gather(3, src), torch.zeros((), device="cuda"))
    b = torch.arange(B, device="cuda")[None, :, None, None].expand_as(src)
    dst = torch.arange(k, device="cuda").expand_as(src)
    lyr, hd = torch.arange(L, device="cuda")[:, None, None, None].expand_as(src), torch.arange(H, device="cuda")[:, None].expand_as(src)
    at = (lyr[there], s["page_table"][b, src // c["page"]].long()[there], (src % c["page"])[there], hd[there])
    to = (lyr[there], s["page_table"][b, dst // c["page"]].long()[there], (dst % c["page"])[there], hd[there])
    for name in ("k_cache", "v_cache"):
        s[name][to] = s[name][at]
    if k < C:
        kept = torch.cat([kept, torch.full((L, B, H, C - k), -1, device="cuda")], 3)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "ctx_len": new_len, "kept": kept.to(torch.int32),
            "weights": wout}


# ---------------------------------------------------------------------------
# the same from the definition, in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------
def _slots(s, b, count):
    """(page, slot) of the first `count` positions of sequence b."""
    n = torch.arange(count, device="cuda")
    ps = s["case"]["page"]
    return s["page_table"][b][n // ps].long(), n % ps


def _hidden(c, L, first, last):
    """[last - first, L + last]: which slots tokens first..last-1 behind L slots do not see."""
    i = torch.arange(first, last, device="cuda")[:, None] + L
    j = torch.arange(L + last, device="cuda")[None, :]
    hide = j > i
    if c["window"]:
        hide |= (i - j >= c["window"]) & (j >= c["sinks"])
    return hide


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    lens = s["ctx_len"].tolist()
    if c["op"] == "evict":
        S, C = s["weights"].shape[3], c["budget"]
        k, v, wout = s["k_cache"].double(), s["v_cache"].double(), torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
        for b, L in enumerate(lens):
            if L <= C:
                wout[:, b, :, :L] = s["weights"][:, b, :, :L].double()
                continue
            pages, offs = _slots(s, b, L)
            for layer in range(c["layers"]):
                for h in range(c["Hkv"]):
                    mid = s["weights"][layer, b, h, c["sinks"]:L - c["recent"]]
                    order = torch.sort(mid, descending=True, stable=True).indices[:C - c["sinks"] - c["recent"]]
                    keep = torch.cat([torch.arange(c["sinks"], device="cuda"), order.sort().values + c["sinks"],
                                      torch.arange(L - c["recent"], L, device="cuda")])
                    wout[layer, b, h, :C] = s["weights"][layer, b, h, keep].double()
                    for new, old in ((k, s["k_cache"]), (v, s["v_cache"])):
                        new[layer, pages[:C], offs[:C], h] = old[layer, pages[keep], offs[keep], h].double()
        return {"k_cache": k, "v_cache": v, "ctx_len": None, "kept": None, "weights": wout}
    N, H, D = c["N"], c["Hkv"], c["D"]
    G = c["Hq"] // H
    counts = [N] * c["B"] if s["n_nodes"] is None else s["n_nodes"].tolist()
    out = torch.zeros((c["B"], N, c["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], N, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    W = s["weights"].double() if c["op"] == "sum" else None
    step = max(1, 150000000 // ((max(lens) + N) * G))  # tokens side by side
    for b, L in enumerate(lens):
        n = counts[b]
        if n == 0:
            continue
        pages, offs = _slots(s, b, L + n)
        if W is not None:
            W[b, :, :L + n] *= c["decay"]
        for h in range(H):
            K = s["k_cache"][:, :, h][pages, offs].double()
            V = s["v_cache"][:, :, h][pages, offs].double()
            for i in range(0, n, step):
                e = min(n, i + step)
                q = s["q"][b, i:e, h * G:(h + 1) * G].double()
                x = torch.einsum("ngd,sd->ngs", q, K[:L + e]) / math.sqrt(D)
                x.masked_fill_(_hidden(c, L, i, e)[:, None, :], -math.inf)
                if W is not None:
                    W[b, h, :L + e] += torch.exp(x - s["lse"][b, i:e, h * G:(h + 1) * G, None].double()).sum((0, 1))
                    continue
                lse[b, i:e, h * G:(h + 1) * G] = torch.logsumexp(x, 2)
                out[b, i:e, h * G:(h + 1) * G] = torch.einsum("ngs,sd->ngd", torch.softmax(x, 2), V[:L + e])
    return {"weights": W} if W is not None else {"out": out, "lse": lse}
