"""Corners of the target pass's operators: temperatures and logits at the ends
of their ranges, masked tokens, workspaces in turn, huge scores, heads that
share a block with many tokens' heads.

Tolerances as in tests/test_gpu_target.py.
"""
import math

import pytest
import torch

import target_reference as ref
from test_gpu_target import BF, FP, _check_attention, _check_logprobs, _same

pytestmark = pytest.mark.gpu


def test_logprobs_extreme_temperatures(gpu_lib):
    """1 / T from 1e9 down to 1e-30: one token takes it all, or all are alike."""
    gen = torch.Generator().manual_seed(31)
    T = torch.tensor([1e-9, 5e-8, 2e-7, 1e-4, 1e4, 1e20, 3e24, 1e30])
    for dt, V in ((torch.float32, 9001), (BF, 20000)):
        z = (torch.randn((8, V), generator=gen) * 3).to(dt)
        z[:, 17] = 40.0  # the best by far: the others' probabilities are 0 where T is small
        tok = torch.tensor([17, 17, 17, 17, 5, 5, 5, 17], dtype=torch.int32)
        for K in (0, 4):
            _check_logprobs(gpu_lib, z.cuda(), tok, K, T)


def test_logprobs_infinite_temperature(gpu_lib):
    """All tokens that are not masked are alike."""
    z = torch.full((1, 30000), -math.inf)
    z[0, ::3] = torch.randn(10000, generator=torch.Generator().manual_seed(32))
    tok = torch.tensor([3], dtype=torch.int32).cuda()
    g = gpu_lib.ssd_logprobs(z.cuda(), tok, 3, torch.tensor([math.inf]).cuda())
    # a sum of 10^4 ones and a logarithm in 32 bits
    assert abs(float(g["logprob"]) + math.log(10000)) <= 2.0 ** -19
    assert abs(float(g["entropy"]) - math.log(10000)) <= 2.0 ** -19


@pytest.mark.parametrize("K", [0, 5])
def test_logprobs_large_logits(gpu_lib, K):
    """m / T beyond 2^24, where the maximum's own product is rounded by more
    than the logits differ; and maxima that grow all along the row."""
    gen = torch.Generator().manual_seed(33)
    V = 40000
    z = torch.zeros((4, V))
    z[0] = 5e7 + 8 * torch.randint(0, 4, (V,), generator=gen)
    z[1] = -5e7 + 8 * torch.randint(0, 4, (V,), generator=gen)
    z[2] = torch.arange(V).float() * 0.25
    z[3] = 3e8 * torch.randn(V, generator=gen)
    tok = torch.tensor([7, 8, V - 3, int(z[3].argmax())], dtype=torch.int32)
    _check_logprobs(gpu_lib, z.cuda(), tok, K)


def test_logprobs_rank_of_masked_and_equal_tokens(gpu_lib):
    V = 5003
    z = torch.randn((3, V), generator=torch.Generator().manual_seed(34))
    z[0, 100:4000] = -math.inf  # masked tokens rank behind all others, by index
    z[1, 50:4500] = 6.0
    z[2, :] = 1.5
    tok = torch.tensor([2100, 4499, 5002], dtype=torch.int32)
    for dt in (torch.float32, BF):
        g = gpu_lib.ssd_logprobs(z.to(dt).cuda(), tok.cuda(), 2)
        assert g["rank"].tolist() == [V - 3900 + 2001, 4450, V]
        assert float(g["logprob"][0]) == -math.inf
        assert g["top_tok"][1:].tolist() == [[50, 51], [0, 1]]


def test_logprobs_workspace_in_turn(gpu_lib):
    """One workspace for calls of different sizes: rows in parts and whole."""
    gen = torch.Generator().manual_seed(35)
    ws = gpu_lib.new_workspace(
        max(gpu_lib.load_library().ssd_logprobs_workspace_bytes(R, 70001, 8) for R in (1, 5, 200)), "cuda")
    calls = []
    for R, K, dt in ((1, 8, BF), (5, 3, torch.float32), (200, 0, BF), (2, 8, torch.float32), (200, 8, BF), (1, 0, BF)):
        z = torch.randn((R, 70001), generator=gen).to(dt).cuda()
        tok = torch.randint(0, 70001, (R,), generator=gen).to(torch.int32).cuda()
        calls.append((z, tok, K))
    alone = [gpu_lib.ssd_logprobs(*a) for a in calls]
    for _ in range(2):
        for a, want in zip(calls, alone):
            got = gpu_lib.ssd_logprobs(*a, ws=ws)
            for key in want:
                if key != "ws":
                    assert torch.equal(got[key], want[key]), key
    assert gpu_lib.get_device_error(ws) == 0


@pytest.mark.parametrize("dt", [BF, FP])
def test_attention_huge_scores(gpu_lib, dt):
    """Scores of thousands: nearly all of a row's weight on one slot, running
    maxima that jump by more than any exponential holds."""
    c = ref.case(2, 6, 8, 2, 128, 16, (300, 901), dt, 36)
    _check_attention(gpu_lib, c, scale=20.0)
    c = ref.case(2, 24, 8, 2, 64, 16, (300, 901), dt, 37)
    _check_attention(gpu_lib, c, scale=-9.0)


@pytest.mark.parametrize("D", [64, 128])
def test_kv_append_small_heads_many_tokens(gpu_lib, D):
    """Three heads a token: a block's range covers many tokens and begins and
    ends inside them."""
    for N, dt in ((1, BF), (7, FP)):
        c = ref.case(300, N, 1, 1, D, 16, tuple(i % 50 for i in range(300)), dt, 38 + N)
        c["cos_sin"] = gpu_lib.rope_table(64, D, device="cpu")
        q, kc, vc, qt, kt = ref.append(c, D)
        g = ref.to_gpu(c)
        r = gpu_lib.ssd_kv_append(g["q"], g["k"], g["v"], g["k_cache"], g["v_cache"], g["page_table"], g["ctx_len"],
                                  parent=g["parent"], cos_sin=g["cos_sin"])
        _same(r["q"], q, qt, "q")
        _same(g["k_cache"], kc, kt, "k_cache")
        assert torch.equal(g["v_cache"].cpu().double(), vc)
        assert gpu_lib.get_device_error(r["ws"]) == 0
