"""Speculative decoding with token trees over a paged cache: a small decoder
of random weights and the calls of a round in the order of a serving loop.

    python examples/tree_decode.py [--tokens 48] [--temperature 0.8] [--batch 4]

A round: the draft grows a tree of tokens below the last committed one; the
target runs once over its nodes (ssd_kv_append and ssd_tree_attention in every
layer); ssd_verify_tree accepts a path; ssd_kv_commit moves its keys and values
behind the context in all layers; ssd_logprobs answers with the emitted tokens'
log probabilities.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_70_gb300 as ssd  # noqa: E402


class Decoder:
    """Pre-norm decoder: grouped queries, normed heads, rotated positions.  Its
    attention adds little to a token's own path, so that the path without
    attention is a draft that is often right."""

    def __init__(self, V=1000, layers=2, dim=256, Hq=8, Hkv=2, D=64, max_pos=4096, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def rand(*shape, std):
            return (torch.randn(shape, generator=g, device=device) * std).to(torch.bfloat16)

        self.V, self.layers, self.Hq, self.Hkv, self.D = V, layers, Hq, Hkv, D
        self.emb = rand(V, dim, std=1.0)
        self.wqkv = [rand(dim, (Hq + 2 * Hkv) * D, std=dim ** -0.5) for _ in range(layers)]
        self.wo = [rand(Hq * D, dim, std=0.5 * (Hq * D) ** -0.5) for _ in range(layers)]
        self.up = [rand(dim, 2 * dim, std=dim ** -0.5) for _ in range(layers)]
        self.down = [rand(2 * dim, dim, std=(2 * dim) ** -0.5) for _ in range(layers)]
        self.head = rand(dim, V, std=3.0 * dim ** -0.5)
        self.q_norm = torch.ones(D, dtype=torch.bfloat16, device=device)
        self.k_norm = torch.ones(D, dtype=torch.bfloat16, device=device)
        self.cos_sin = ssd.rope_table(max_pos, D, device=device)

    @staticmethod
    def _norm(x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def _logits(self, x):
        return (self._norm(x) @ self.head).float()

    def _mlp(self, x, i):
        return (torch.nn.functional.silu(self._norm(x) @ self.up[i]) @ self.down[i]).float()

    def draft(self, tok):
        """Logits without attention."""
        x = self.emb[tok.long()].float()
        for i in range(self.layers):
            x = x + self._mlp(x, i)
        return self._logits(x)

    def forward(self, tok, cache, parent=None, n_nodes=None):
        """Logits [B, N, V] at the nodes tok [B, N] behind the cache's contexts."""
        B, N = tok.shape
        x = self.emb[tok.long()].float()
        for i in range(self.layers):
            qkv = (self._norm(x) @ self.wqkv[i]).view(B, N, self.Hq + 2 * self.Hkv, self.D)
            q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], dim=2)
            at = (cache.k[i], cache.v[i], cache.table, cache.ctx_len)
            a = ssd.ssd_kv_append(q, k, v, *at, parent=parent, n_nodes=n_nodes, cos_sin=self.cos_sin,
                                  q_norm=self.q_norm, k_norm=self.k_norm, ws=cache.ws.get("append"))
            o = ssd.ssd_tree_attention(a["q"], *at, parent=parent, n_nodes=n_nodes, ws=cache.ws.get((B, N)))
            cache.ws["append"], cache.ws[B, N] = a["ws"], o["ws"]
            x = x + (o["out"].reshape(B, N, -1) @ self.wo[i]).float()
            x = x + self._mlp(x, i)
        return self._logits(x)


class PagedCache:
    """Keys and values of all layers in pages of `ps` slots, `length` slots a
    sequence; the pages in no order, as an allocator would leave them."""

    def __init__(self, model, B, length, ps=16, seed=0):
        dev = model.emb.device
        width = -(-length // ps)
        shape = (model.layers, B * width, ps, model.Hkv, model.D)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
        self.v = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
        g = torch.Generator()
        g.manual_seed(seed)
        self.table = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width).to(dev)
        self.ctx_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.ws = {}

    def commit(self, accept_len, out_node=None):
        r = ssd.ssd_kv_commit(self.k, self.v, self.table, self.ctx_len, accept_len, out_node, ws=self.ws.get("commit"))
        self.ctx_len, self.ws["commit"] = r["ctx_len"], r["ws"]

    def errors(self):
        return {name: ssd.get_device_error(ws) for name, ws in self.ws.items()}


def tree_parents(widths):
    """Parents of a tree with widths[d] children a node at depth d."""
    par, level = [-1], [0]
    for w in widths:
        level = [(par.append(p), len(par) - 1)[1] for p in level for _ in range(w)]
    return par


def prefill(model, cache, prompt, chunk=64):
    """The prompt [B, n] into the cache, as chains of up to 64 nodes; no moves,
    so the commit only moves the lengths."""
    for at in range(0, prompt.shape[1], chunk):
        part = prompt[:, at:at + chunk].contiguous()
        model.forward(part, cache)
        cache.commit(torch.full((part.shape[0],), part.shape[1] - 1, dtype=torch.int32, device=part.device))


def grow_tree(model, root, widths, T, gen):
    """A tree below root [B]: children drawn from the draft's law at their
    parent (the most likely ones where T is 0).  Returns tok [B, N], D [B, N, V]."""
    toks, laws, level = [root[:, None]], [], root[:, None]
    for w in widths:
        d = model.draft(level)
        laws.append(d)
        p = torch.softmax(d / T.clamp(min=1e-6)[:, None, None], -1).flatten(0, 1)
        drawn = torch.multinomial(p, w, replacement=True, generator=gen)
        best = d.flatten(0, 1).topk(w, dim=-1).indices
        greedy = (T == 0)[:, None].expand(level.shape).reshape(-1, 1)
        level = torch.where(greedy, best, drawn).view(root.shape[0], -1).to(torch.int32)
        toks.append(level)
    laws.append(torch.zeros_like(laws[0][:, :1]).expand(-1, level.shape[1], -1))  # (leaves: not read)
    return torch.cat(toks, 1).contiguous(), torch.cat(laws, 1).contiguous()


def decode(model, prompt, tokens, widths=(3, 2, 1), temperature=0.0, top=0, seed=0):
    """At least `tokens` tokens behind every prompt [B, n].  Returns a dict: for
    every sequence its tokens, their log probabilities under the target at the
    temperature, the tokens a round; and the calls' device error words."""
    B, dev = prompt.shape[0], prompt.device
    par = tree_parents(widths)
    N = len(par)
    parent = torch.tensor(par, dtype=torch.int32, device=dev).expand(B, N).contiguous()
    cache = PagedCache(model, B, prompt.shape[1] + tokens + 2 * N + len(widths))
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    T = torch.full((B,), float(temperature), device=dev)
    prefill(model, cache, prompt[:, :-1])
    limit = prompt.shape[1] + tokens
    root = prompt[:, -1].contiguous()
    out = [[] for _ in range(B)]
    logp = [[] for _ in range(B)]
    rounds = 0
    first = torch.arange(B, device=dev, dtype=torch.int32)[:, None] * N
    while min(len(o) for o in out) < tokens:
        tok, D = grow_tree(model, root, widths, T, gen)
        # sequences that have their tokens stay as they are
        n_nodes = torch.where(cache.ctx_len < limit, N, 0).to(torch.int32)
        Z = model.forward(tok, cache, parent, n_nodes)
        u = torch.rand((B, N + 1), generator=gen, device=dev)
        t = ssd.ssd_verify_tree(Z, D, parent, tok, T, u[:, :N].contiguous(), u[:, N].contiguous(),
                                ws=cache.ws.get("verify"))
        acc = torch.where(n_nodes > 0, t["accept_len"], -1).to(torch.int32)
        cache.commit(acc, t["out_node"])
        # answer i was decided at the path's node i: the root, then the accepted nodes
        path = torch.cat([torch.zeros_like(first), t["out_node"][:, :-1]], 1)
        rows = torch.where(torch.arange(N, device=dev) <= acc[:, None], first + path, -1).to(torch.int32)
        a = ssd.ssd_logprobs(Z.view(B * N, -1), t["out_tok"].view(-1), top, T.repeat_interleave(N), rows=rows.view(-1),
                             ws=cache.ws.get("logprobs"))
        cache.ws["verify"], cache.ws["logprobs"] = t["ws"], a["ws"]
        root = torch.where(acc >= 0, t["out_tok"].gather(1, acc.clamp(min=0).long()[:, None])[:, 0], root)
        for b, n in enumerate(acc.tolist()):
            out[b] += t["out_tok"][b, :n + 1].tolist()
            logp[b] += a["logprob"].view(B, N)[b, :n + 1].tolist()
        rounds += 1
    return {"tokens": out, "logprob": logp, "a_round": sum(map(len, out)) / (B * rounds), "errors": cache.errors()}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--tokens", type=int, default=48)
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--batch", type=int, default=4)
    args = ap.parse_args()
    model = Decoder()
    prompt = torch.randint(0, model.V, (args.batch, 20), dtype=torch.int32, device="cuda")
    r = decode(model, prompt, args.tokens, temperature=args.temperature)
    for tok, lp in zip(r["tokens"], r["logprob"]):
        print(" ".join("%d" % t for t in tok[:16]), "...  mean log probability %.3f" % (sum(lp) / len(lp)))
    print("%.2f tokens a sequence and round; device errors: %s"
          % (r["a_round"], {k: v for k, v in r["errors"].items() if v} or "none"))


if __name__ == "__main__":
    main()
