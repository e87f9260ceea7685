"""Log probabilities at the ends of their range: rows of the type's lowest
value, tokens there, infinite temperatures and ones without a reciprocal, and rows of
which one token takes nearly all.

Tolerances as in tests/test_gpu_target.py; what exceeds 32 bits is infinite.
"""
import math

import pytest
import torch

import target_reference as ref
from test_gpu_target import BF, _check_logprobs, _same

pytestmark = pytest.mark.gpu
F32 = torch.float32
# (rows, V): whole rows, a row in parts, an odd length
SIZES = [(5, 3001), (2, 70001), (3, 128256)]


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("K", [0, 4])
def test_rows_of_the_lowest_values(gpu_lib, dt, K):
    """Rows whose finite logits all lie at or below -3e38 are rows like others."""
    low = torch.finfo(dt).min
    for R, V in SIZES:
        z = torch.full((R, V), low).to(dt)
        z[1, ::2] = -math.inf                      # and half of them masked
        if R > 2:
            z[2, V // 3] = -3.1e38                 # one token far above the others
        tok = torch.tensor([7, 1, V // 3, 0, V - 1][:R], dtype=torch.int32)
        _check_logprobs(gpu_lib, z.cuda(), tok, K)
        _check_logprobs(gpu_lib, z.cuda(), tok, K, torch.linspace(0.3, 40.0, R))


@pytest.mark.parametrize("dt", [F32, BF])
def test_greedy_rows_of_the_lowest_value(gpu_lib, dt):
    """T = 0: the one-hot at the lowest index."""
    z = torch.full((2, 9000), torch.finfo(dt).min, dtype=dt)
    g = gpu_lib.ssd_logprobs(z.cuda(), torch.tensor([0, 5], dtype=torch.int32).cuda(), 2, torch.zeros(2).cuda())
    assert g["logprob"].tolist() == [0.0, -math.inf] and g["entropy"].tolist() == [0.0, 0.0]
    assert g["rank"].tolist() == [1, 6] and g["top_tok"].tolist() == [[0, 1]] * 2
    assert gpu_lib.get_device_error(g["ws"]) == 0


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("V", [500, 70001])
def test_tokens_of_the_lowest_value(gpu_lib, dt, V):
    """A token at the type's lowest value among ordinary ones: about -3.4e38 / T,
    -inf only where that exceeds 32 bits.  And one that lies further below the
    best than 32 bits hold, at a T that brings it back."""
    low = torch.finfo(dt).min
    z = torch.randn((4, V), generator=torch.Generator().manual_seed(41)).to(dt)
    z[:, 3] = low
    z[3, 9] = -low
    T = torch.tensor([1.0, 2.5, 0.9, 4.0])
    tok = torch.tensor([3, 3, 3, 3], dtype=torch.int32)
    lp, H, rank, _, _ = ref.logprobs(z, tok, 1, T)
    g = gpu_lib.ssd_logprobs(z.cuda(), tok.cuda(), 0, T.cuda())
    _same(g["logprob"], lp.float().double(), lp.abs().clamp(max=1e300) * 2.0 ** -21, "logprob")
    assert g["rank"].tolist() == rank.tolist() == [V] * 4
    few = z[:, :20].contiguous()  # all of them asked for
    lp, H, rank, top, tlp = ref.logprobs(few, tok, 20, T)
    g = gpu_lib.ssd_logprobs(few.cuda(), tok.cuda(), 20, T.cuda())
    assert torch.equal(g["top_tok"].cpu().long(), top)
    _same(g["top_logprob"], tlp.float().double(), 2.0 ** -19 + tlp.abs() * 2.0 ** -21, "top_logprob")
    assert gpu_lib.get_device_error(g["ws"]) == 0


@pytest.mark.parametrize("dt", [F32, BF])
def test_masked_tokens_at_infinite_temperature(gpu_lib, dt):
    """All that are not masked are alike; masked ones have no probability."""
    z = torch.full((2, 6000), -math.inf, dtype=dt)
    z[0, 5:8] = torch.tensor([1.0, -2.0, 0.5]).to(dt)
    z[1, [9, 77]] = torch.tensor([torch.finfo(dt).max, torch.finfo(dt).min], dtype=dt)
    tok = torch.tensor([4, 77], dtype=torch.int32)
    g = gpu_lib.ssd_logprobs(z.cuda(), tok.cuda(), 6, torch.full((2,), math.inf).cuda())
    n = torch.tensor([3.0, 2.0], dtype=torch.float64)
    want = torch.full((2, 6), -math.inf, dtype=torch.float64)
    want[0, :3], want[1, :2] = -math.log(3), -math.log(2)
    _same(g["top_logprob"], want, torch.full_like(want, 2.0 ** -20), "top_logprob")
    _same(g["logprob"], torch.tensor([-math.inf, -math.log(2)], dtype=torch.float64), torch.full((2,), 2.0 ** -20), "logprob")
    _same(g["entropy"], n.log(), torch.full((2,), 2.0 ** -20, dtype=torch.float64), "entropy")
    assert g["top_tok"].tolist() == [[5, 7, 6, 0, 1, 2], [9, 77, 0, 1, 2, 3]]
    assert g["rank"].tolist() == [8, 2]
    assert gpu_lib.get_device_error(g["ws"]) == 0


def test_differences_beyond_32_bits(gpu_lib):
    """Logits further apart than 32 bits hold, at temperatures that bring them
    near again: in one part of a row, and in several."""
    for V in (2000, 128256):
        z = torch.zeros((2, V))
        z[:, 3], z[:, V - 2] = torch.finfo(F32).max, torch.finfo(F32).min
        z[1, V // 2:] = torch.finfo(F32).min
        tok = torch.tensor([V - 2, V - 1], dtype=torch.int32)
        for K in (0, 3):
            _check_logprobs(gpu_lib, z.cuda(), tok, K, torch.tensor([2e38, 1.5e38]))


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("K", [0, 3])
def test_temperatures_without_reciprocal(gpu_lib, dt, K):
    """log2(e) / T beyond 32 bits: the best share everything, equally; and
    logits that are as small as T."""
    for R, V in ((3, 4001), (3, 70001)):
        z = torch.randn((R, V), generator=torch.Generator().manual_seed(42)).to(dt)
        z[0, [40, 1999]] = 9.0
        z[1, 7] = 9.0
        T = torch.tensor([1e-40, 3e-39, 2e-45])
        tok = torch.tensor([1999, 7, 11], dtype=torch.int32)
        lp, H, rank, top, tlp = ref.logprobs(z, tok, max(K, 1), T)
        g = gpu_lib.ssd_logprobs(z.cuda(), tok.cuda(), K, T.cuda())
        _same(g["logprob"], lp.float().double(), torch.full_like(lp, 2.0 ** -20), "logprob")
        _same(g["entropy"], H, torch.full_like(H, 2.0 ** -20), "entropy")
        assert torch.equal(g["rank"].cpu().long(), rank.long())
        if K:
            assert torch.equal(g["top_tok"].cpu().long(), top)
            _same(g["top_logprob"], tlp.float().double(), torch.full_like(tlp, 2.0 ** -20), "top_logprob")
        assert gpu_lib.get_device_error(g["ws"]) == 0
    z = torch.zeros((1, 64))
    z[0, 5:9] = torch.tensor([1.0, 2.0, 3.0, 0.5]) * 1e-39
    _check_logprobs(gpu_lib, z.cuda(), torch.tensor([6], dtype=torch.int32), K, torch.tensor([5e-40]))


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("K", [0, 2])
@pytest.mark.parametrize("R,V", [(1500, 4097), (40, 70001)])
def test_no_probability_above_one(gpu_lib, dt, K, R, V):
    """One token takes all but 1e-9, others share the rest or there is none: a log
    probability is at most 0 and an entropy at least 0."""
    gen = torch.Generator().manual_seed(43)
    z = torch.randn((R, V), generator=gen)
    best = torch.randint(0, V, (R,), generator=gen)
    z[torch.arange(R), best] = 30 + 40 * torch.rand(R, generator=gen)
    z = (z + 60 * torch.rand((R, 1), generator=gen)).to(dt)
    tok = z.float().argmax(1).to(torch.int32)
    T = 0.2 + torch.rand(R, generator=gen)
    for t in (T, torch.ones(R)):
        g = _check_logprobs(gpu_lib, z.cuda(), tok, K, t)
        assert float(g["logprob"].max()) <= 0.0 and float(g["entropy"].min()) >= 0.0
        if K:
            assert float(g["top_logprob"].max()) <= 0.0
