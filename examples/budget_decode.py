"""Decoding with a cache of a fixed budget: a small decoder of random weights, and
the calls in the order of a serving loop.

    python examples/budget_decode.py [--prompt 700] [--tokens 64] [--budget 256] [--batch 4]

The prompt goes in by chunks (ssd_kv_append and ssd_chunk_attention in every layer).
Its last tokens, and every decoded one, add their attention weights up for each slot
(ssd_kv_weights); whenever a cache has grown past its budget, every head keeps its
heaviest slots, the first and the latest tokens (ssd_kv_evict).  Kept keys stay turned
by the positions of their tokens, and new ones go by their positions, not their slots.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_70_gb300 as ssd  # noqa: E402
from examples.tree_decode import Decoder, PagedCache  # noqa: E402


class BudgetedCache(PagedCache):
    """A paged cache with the weights of its slots, and how many tokens each sequence
    has had (the next token's position)."""

    def __init__(self, model, B, length, budget, sinks=4, recent=32, decay=0.95, **kw):
        super().__init__(model, B, length, **kw)
        self.weights = torch.zeros((model.layers, B, model.Hkv, self.table.shape[1] * self.k.shape[2]),
                                   device=self.k.device)
        self.pos = torch.zeros_like(self.ctx_len)
        self.budget, self.sinks, self.recent, self.decay = budget, sinks, min(recent, budget - sinks), decay

    def cut(self):
        r = ssd.ssd_kv_evict(self.k, self.v, self.table, self.ctx_len, self.weights, self.budget, sinks=self.sinks,
                             recent=self.recent, ws=self.ws.get("evict"), out={"weights": self.weights})
        self.ctx_len, self.ws["evict"] = r["ctx_len"], r["ws"]


def forward(model, tok, cache, observers):
    """Logits [B, V] behind the last of the tokens tok [B, N], which join the cache; its
    last `observers` tokens add their weights."""
    B, N = tok.shape
    x = model.emb[tok.long()].float()
    for i in range(model.layers):
        qkv = (model._norm(x) @ model.wqkv[i]).view(B, N, model.Hq + 2 * model.Hkv, model.D)
        q, k, v = qkv.split([model.Hq, model.Hkv, model.Hkv], dim=2)
        at = (cache.k[i], cache.v[i], cache.table, cache.ctx_len)
        a = ssd.ssd_kv_append(q, k, v, *at, cos_sin=model.cos_sin, q_norm=model.q_norm, k_norm=model.k_norm,
                              pos=cache.pos, ws=cache.ws.get("append"))
        o = ssd.ssd_chunk_attention(a["q"], *at, ws=cache.ws.get((B, N)))
        cache.ws["append"], cache.ws[B, N] = a["ws"], o["ws"]
        n = min(N, observers)
        if n:
            w = ssd.ssd_kv_weights(a["q"][:, N - n:], cache.k[i], cache.table, cache.ctx_len + (N - n),
                                   o["lse"][:, N - n:].contiguous(), cache.weights[i], decay=cache.decay,
                                   ws=cache.ws.get("weights"))
            cache.ws["weights"] = w["ws"]
        x = x + (o["out"].reshape(B, N, -1) @ model.wo[i]).float()
        x = x + model._mlp(x, i)
    cache.ctx_len, cache.pos = cache.ctx_len + N, cache.pos + N
    return model._logits(x[:, -1])


def decode(model, prompt, tokens, budget, spare=32, chunk=256, observers=32):
    """The most likely `tokens` tokens behind every prompt [B, n], with caches that are cut
    to `budget` slots whenever they hold `spare` more.  Returns a dict: tokens [B, tokens],
    the most slots a cache held while decoding, and the calls' device error words."""
    B, n = prompt.shape
    cache = BudgetedCache(model, B, max(n, budget) + spare + 1, budget)
    for at in range(0, n, chunk):
        z = forward(model, prompt[:, at:at + chunk], cache, observers if at + chunk >= n else 0)
    out, held, most = [], n, 0
    for _ in range(tokens):
        if held >= budget + spare or (not out and held > budget):
            cache.cut()
            held = budget
        tok = z.argmax(-1)[:, None].to(torch.int32)
        out.append(tok)
        z = forward(model, tok, cache, 1)
        held += 1
        most = max(most, held)
    assert cache.ctx_len.tolist() == [held] * B
    return {"tokens": torch.cat(out, 1), "slots": most, "errors": cache.errors()}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--budget", type=int, default=256)
    ap.add_argument("--batch", type=int, default=4)
    args = ap.parse_args()
    model = Decoder()
    prompt = torch.randint(0, model.V, (args.batch, args.prompt), dtype=torch.int32, device="cuda")
    r = decode(model, prompt, args.tokens, args.budget)
    for tok in r["tokens"].tolist():
        print(" ".join("%d" % t for t in tok[:16]), "...")
    print("%d slots at most; device errors: %s" % (r["slots"], {k: v for k, v in r["errors"].items() if v} or "none"))


if __name__ == "__main__":
    main()
