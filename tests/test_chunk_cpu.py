"""What the operators of prompts and budgets refuse, at the C entry points and in the binding,
and their plain forms against hand-made cases.  Nothing is launched."""
import math

import pytest
import torch

import chunk_reference as cref
import target_reference as ref
from speculative_decoding_verification_70_gb300 import _binding as bd
from test_abi_cpu import lib, needs_no_gpu  # noqa: F401
from test_target_binding_cpu import I32, Launched, OnOtherGpu, _ws, gpu, no_launch  # noqa: F401
from test_target_cpu import BAD_KV, DTYPE, INVALID, P, WORKSPACE, _kv, _nodes

BF = torch.bfloat16
BAD_TOKENS = [dict(B=0), dict(N=0), dict(N=(1 << 20) + 1), dict(ctx_len=None), dict(parent=P), dict(n_nodes=P + 2),
              dict(B=1 << 30), dict(B=4096, N=1 << 20)]


def _attend(lib, kv=None, tokens=None, Hq=16, q=P, q_b=4 * 16 * 128, q_n=16 * 128, q_h=128, window=5, sinks=1, scale=0.1,
            out=P, lse=P, ws=P, n=1 << 40):
    return lib.ssd_chunk_attention(kv or _kv(), tokens or _nodes(), Hq, q, q_b, q_n, q_h, window, sinks, scale, out,
                                   lse, ws, n, None)


def _sum(lib, kv=None, tokens=None, Hq=16, q=P, q_b=4 * 16 * 128, q_n=16 * 128, q_h=128, lse=P, window=5, sinks=1,
         scale=0.1, decay=1.0, w=P, w_b=8 * 64, w_h=64, w_len=64, ws=P, n=1 << 40):
    return lib.ssd_kv_weights(kv or _kv(), tokens or _nodes(), Hq, q, q_b, q_n, q_h, lse, window, sinks, scale, decay, w,
                              w_b, w_h, w_len, ws, n, None)


def _evict(lib, kv=None, layers=2, kl=1 << 20, vl=1 << 20, B=2, ctx=P, w=P, w_l=1024, w_b=512, w_h=64, w_len=64,
           budget=32, sinks=4, recent=8, new=P + 64, kept=P, wo=P, wo_l=1024, wo_b=512, wo_h=64, ws=P, n=256):
    return lib.ssd_kv_evict(kv or _kv(), layers, kl, vl, B, ctx, w, w_l, w_b, w_h, w_len, budget, sinks, recent, new,
                            kept, wo, wo_l, wo_b, wo_h, ws, n, None)


@needs_no_gpu
@pytest.mark.parametrize("kw", BAD_KV, ids=str)
def test_bad_cache_is_refused(lib, kw):
    for call in (_attend, _sum, _evict):
        assert call(lib, kv=_kv(**kw)) == INVALID


@needs_no_gpu
@pytest.mark.parametrize("kw", BAD_TOKENS, ids=str)
def test_bad_tokens_are_refused(lib, kw):
    for call in (_attend, _sum):
        assert call(lib, tokens=_nodes(**kw)) == INVALID


@needs_no_gpu
def test_attention_refusals(lib):
    assert _attend(lib, kv=_kv(dtype=0)) == DTYPE
    for kw in (dict(Hq=12), dict(Hq=4), dict(Hq=8 * 65), dict(q=None), dict(q=P + 8), dict(q_n=1028), dict(q_b=0),
               dict(q_h=-128), dict(q_b=1 << 38), dict(window=-1), dict(sinks=-1), dict(scale=math.nan),
               dict(scale=math.inf), dict(scale=2.1e38), dict(out=None), dict(out=P + 8), dict(lse=P + 2), dict(ws=None),
               dict(ws=P + 16)):
        assert _attend(lib, **kw) == INVALID, kw
    need = lib.ssd_chunk_attention_workspace_bytes(2, 4, 16, 8, 128)
    assert need >= 256 and _attend(lib, n=need - 1) == WORKSPACE
    for a in ((0, 1, 1, 1, 64), (1, (1 << 20) + 1, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 1, 1, 80), (1, 1, 65, 1, 64)):
        assert lib.ssd_chunk_attention_workspace_bytes(*a) == 0


@needs_no_gpu
def test_weights_refusals(lib):
    assert _sum(lib, kv=_kv(dtype=0)) == DTYPE
    for kw in (dict(Hq=12), dict(Hq=8 * 65), dict(q=None), dict(q=P + 8), dict(q_h=1028), dict(q_n=0), dict(lse=None),
               dict(lse=P + 2), dict(window=-1), dict(sinks=-1), dict(scale=math.inf), dict(decay=math.nan), dict(w=None),
               dict(w=P + 2), dict(w_len=0), dict(w_b=63), dict(w_h=63), dict(w_b=1 << 38), dict(ws=None),
               dict(ws=P + 64)):
        assert _sum(lib, **kw) == INVALID, kw
    need = lib.ssd_kv_weights_workspace_bytes()
    assert need >= 256 and _sum(lib, n=need - 1) == WORKSPACE


@needs_no_gpu
def test_evict_refusals(lib):
    assert _evict(lib, kv=_kv(dtype=0)) == DTYPE
    for kw in (dict(layers=0), dict(kl=4), dict(vl=0), dict(B=0), dict(ctx=None), dict(ctx=P + 2), dict(w=None),
               dict(w_len=0), dict(w_l=63), dict(w_b=63), dict(w_h=63), dict(wo_l=63), dict(wo_b=63), dict(wo_h=63),
               dict(budget=0), dict(sinks=-1), dict(recent=-1), dict(sinks=20, recent=13), dict(new=None), dict(new=P),
               dict(new=P + 4), dict(kept=None), dict(kept=P + 2), dict(wo=P + 4), dict(wo=P + 2), dict(wo_h=128),
               dict(wo=P + 8000), dict(ws=None), dict(layers=1 << 20, B=1 << 20),
               dict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1)):
        assert _evict(lib, **kw) == INVALID, kw
    assert _evict(lib, n=8) == WORKSPACE


@needs_no_gpu
def test_append_of_chains_and_positions_refusals(lib):
    def call(tokens, pos0=P):
        return lib.ssd_kv_append_at(_kv(), tokens, pos0, 16, P, 99, 128, 128, P, P, 512, 128, 128, P, P, 99, 128, 0, P,
                                    P, 1e-6, P, 255, None)
    for kw in (dict(N=65, parent=P), dict(B=0), dict(N=(1 << 20) + 1), dict(ctx_len=None)):
        assert call(_nodes(**kw)) == INVALID, kw
    assert call(_nodes(), P + 2) == INVALID
    for kw in (dict(N=65), dict(N=1 << 20), dict(N=64, parent=P)):  # (the workspace is too small)
        assert call(_nodes(**kw)) == WORKSPACE, kw


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def _case(N=3):
    c = ref.case(2, N, 4, 2, 64, 16, (5, 20), BF, 1, tree="chain")
    return {k: gpu(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def _calls(c, kind=None, **other):
    """The three calls with some tensors replaced."""
    t = dict(q=c["q"], k=c["k_cache"], v=c["v_cache"], table=c["page_table"], ctx=c["ctx_len"],
             n=gpu(torch.zeros(2, dtype=I32)), lse=gpu(torch.zeros(2, c["N"], 4)), w=gpu(torch.zeros(2, 2, 50)), ws=_ws(),
             out=gpu(torch.empty((2, c["N"], 4, 64), dtype=BF)), olse=gpu(torch.empty((2, c["N"], 4))),
             new=gpu(torch.empty(2, dtype=I32)), kept=gpu(torch.empty((2, 2, 7), dtype=I32)),
             wo=gpu(torch.empty(2, 2, 50)))
    used = [{"q", "k", "v", "table", "ctx", "n", "ws", "out", "olse"}, {"q", "k", "table", "ctx", "n", "lse", "w", "ws"},
            {"k", "v", "table", "ctx", "w", "ws", "new", "kept", "wo"}]
    t.update(other)
    return used, [
        lambda: bd.ssd_chunk_attention(t["q"], t["k"], t["v"], t["table"], t["ctx"], n_nodes=t["n"], ws=t["ws"],
                                       out={"out": t["out"], "lse": t["olse"]}),
        lambda: bd.ssd_kv_weights(t["q"], t["k"], t["table"], t["ctx"], t["lse"], t["w"], n_nodes=t["n"], ws=t["ws"]),
        lambda: bd.ssd_kv_evict(t["k"], t["v"], t["table"], t["ctx"], t["w"], 7, sinks=1, recent=2, ws=t["ws"],
                                out={"ctx_len": t["new"], "kept": t["kept"], "weights": t["wo"]})], t


@needs_no_gpu
def test_calls_that_fit_reach_the_library(no_launch):  # noqa: F811
    for N in (3, 70):
        _, calls, _ = _calls(_case(N))
        for call in calls:
            with pytest.raises(Launched):
                call()


BAD = [dict(q=torch.zeros(2, 3, 4, 64)), dict(q=torch.zeros(2, 3, 4, 32, dtype=BF)), dict(k=torch.zeros(9, 16, 2, 64)),
       dict(table=torch.zeros(2, 3)), dict(ctx=torch.zeros(3, dtype=I32)), dict(ctx=torch.zeros(2)),
       dict(n=torch.zeros(3, dtype=I32)), dict(lse=torch.zeros(2, 3, 2)), dict(lse=torch.zeros(2, 3, 4, dtype=BF)),
       dict(lse=torch.zeros(2, 4, 3).transpose(1, 2)), dict(w=torch.zeros(2, 3, 50)), dict(w=torch.zeros(2, 2, 50, dtype=BF)),
       dict(w=torch.zeros(2, 50, 2).transpose(1, 2)), dict(out=torch.empty(2, 3, 4, 64)), dict(olse=torch.empty(2, 3, 2)),
       dict(new=torch.empty(3, dtype=I32)), dict(kept=torch.empty((2, 2, 6), dtype=I32)), dict(kept=torch.empty(2, 2, 7)),
       dict(wo=torch.empty(2, 2, 51)), dict(wo=torch.empty(2, 1, 50))]


@needs_no_gpu
@pytest.mark.parametrize("kw", BAD, ids=lambda d: "-".join("%s%s" % (k, list(v.shape)) for k, v in d.items()))
def test_wrong_sizes_and_types(no_launch, kw):  # noqa: F811
    (name, t), = kw.items()
    used, calls, _ = _calls(_case(), **{name: gpu(t)})
    for names, call in zip(used, calls):
        if name in names:
            with pytest.raises((TypeError, ValueError)):
                call()


@needs_no_gpu
def test_tensors_of_another_device(no_launch):  # noqa: F811
    used, _, t = _calls(_case())
    for name in sorted(set().union(*used)):
        _, calls, _ = _calls(_case(), **{name: torch.Tensor._make_subclass(OnOtherGpu, t[name].as_subclass(torch.Tensor))})
        for names, call in zip(used, calls):
            if name in names:
                with pytest.raises(ValueError):
                    call()


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def test_which_slots_are_seen():
    assert cref.seen(2, 3, 0, 0).int().tolist() == [[1, 1, 1, 0, 0], [1, 1, 1, 1, 0], [1, 1, 1, 1, 1]]
    assert cref.seen(2, 3, 2, 0).int().tolist() == [[0, 1, 1, 0, 0], [0, 0, 1, 1, 0], [0, 0, 0, 1, 1]]
    assert cref.seen(2, 3, 1, 2).int().tolist() == [[1, 1, 1, 0, 0], [1, 1, 0, 1, 0], [1, 1, 0, 0, 1]]


def test_plain_chunk_is_the_tree_form_of_a_chain():
    c = ref.case(3, 9, 4, 2, 64, 16, (0, 7, 40), BF, 3, tree="chain", ragged=True)
    for a, b in zip(cref.attention(c)[:2], ref.attention(c)[:2]):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-14)


def test_plain_weights_are_the_softmax_summed():
    c = ref.case(1, 3, 2, 2, 64, 16, 2, BF, 4, tree="chain")
    _, lse, _, _ = cref.attention(c, window=2)
    w, _ = cref.weights(c, lse, torch.ones(1, 2, 7), window=2, decay=0.5)
    K = cref.gather(c, 0, 5, c["k_cache"])
    for h in range(2):
        want = torch.full((7,), 0.5, dtype=torch.float64)
        want[5:] = 1
        for i, s in enumerate(([1, 2], [2, 3], [3, 4])):
            want[s] += torch.softmax(K[s, h] @ c["q"][0, i, h].double() / 8, 0)
        assert torch.allclose(w[0, h], want, rtol=1e-12)


def test_plain_order_of_weights():
    w = torch.tensor([1.0, math.nan, -0.0, 0.0, 2.0, 1.0, -math.inf, math.inf])
    assert cref.order_of(w) == [7, 4, 0, 5, 2, 3, 6, 1]


def test_plain_eviction_by_hand():
    c = ref.case(1, 1, 1, 1, 64, 4, 9, BF, 5, tree="chain")
    c["ctx_len"][0] = 9
    for n in ("k_cache", "v_cache"):
        c[n] = c[n][None]
    w = torch.tensor([0.0, 1, 5, 1, 7, 1, 0, 9, 2]).view(1, 1, 1, 9)
    k, v, new, kept, wout = cref.evict(c, w, 5, 1, 1)
    assert new.tolist() == [5] and kept.flatten().tolist() == [0, 2, 4, 7, 8]
    assert wout.flatten().tolist() == [0, 5, 7, 9, 2, 0, 0, 0, 0]
    at = lambda t, s: t[0, int(c["page_table"][0, s // 4]), s % 4, 0]  # noqa: E731
    for r, s in enumerate([0, 2, 4, 7, 8]):
        assert torch.equal(at(k, r), at(c["k_cache"], s)) and torch.equal(at(v, r), at(c["v_cache"], s))
    assert torch.equal(at(k, 6), at(c["k_cache"], 6))


@needs_no_gpu
def test_cuts_that_count_beyond_32_bits_are_refused(lib):
    big = 2 ** 31 - 65536
    assert _evict(lib, budget=big) == INVALID
    assert _evict(lib, layers=1, w_l=big, w_b=big, w_h=big, w_len=big, wo=None) == INVALID
