"""The example's rounds: what tree decoding emits is what the target alone says."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import tree_decode as ex  # noqa: E402


def test_tree_parents():
    assert ex.tree_parents((2, 2)) == [-1, 0, 0, 1, 1, 2, 2]
    assert ex.tree_parents((3, 2, 1)) == [-1, 0, 0, 0, 1, 1, 2, 2, 3, 3, 4, 5, 6, 7, 8, 9]


def _alone(model, prompt, tokens):
    """Logits [n, V] before each of the tokens, by chains over a new cache."""
    seq = torch.cat([prompt, torch.tensor(tokens, dtype=torch.int32, device=prompt.device)])[None, :-1]
    cache = ex.PagedCache(model, 1, seq.shape[1], ps=32, seed=5)
    z = []
    for at in range(0, seq.shape[1], 13):
        part = seq[:, at:at + 13].contiguous()
        z.append(model.forward(part, cache)[0])
        cache.commit(torch.full((1,), part.shape[1] - 1, dtype=torch.int32, device=seq.device))
    assert not any(cache.errors().values())
    return torch.cat(z)[len(prompt) - 1:]


# Two passes over the same tokens round the same values to 16 bits (about ten
# times a layer, two layers, and twice at the end), each pass off by half a step
# of 2^-8: at most 22 * 2^-8 of a logit's deviation (3) between them.
TOL = 22 * 2.0 ** -8 * 3


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_tree_decoding_is_the_targets(gpu_lib, temperature):
    model = ex.Decoder()
    gen = torch.Generator().manual_seed(7)
    prompt = torch.randint(0, model.V, (3, 70), generator=gen).to(torch.int32).cuda()
    r = ex.decode(model, prompt, 24, temperature=temperature, seed=3)
    assert not any(r["errors"].values())
    assert r["a_round"] > 1.0  # drafts are accepted
    for b in range(3):
        tok = r["tokens"][b]
        z = _alone(model, prompt[b], tok)
        at = z.gather(1, torch.tensor(tok, device="cuda")[:, None])[:, 0]
        if temperature == 0:
            assert bool((z.max(1).values - at <= TOL).all())
        else:
            want = torch.log_softmax(z.double() / temperature, 1).gather(1, torch.tensor(tok, device="cuda")[:, None])[:, 0]
            got = torch.tensor(r["logprob"][b], dtype=torch.float64, device="cuda")
            assert float((got - want).abs().max()) <= 2 * TOL / temperature
