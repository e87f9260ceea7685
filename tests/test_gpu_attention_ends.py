"""Tree attention at the ends of its range: values near the type's largest, and
small ones.

Tolerances as in tests/test_gpu_target.py.
"""
import pytest
import torch

import target_reference as ref
from test_gpu_target import BF, FP, _check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,D", [(1, 64), (6, 128), (40, 64)])
def test_large_values(gpu_lib, N, D):
    """Values near the type's largest, of which the result is a mean: finite,
    wherever the running maximum stands and however many slots share."""
    for dt in (BF, FP):
        c = ref.case(2, N, 4, 2, D, 16, (300, 1500), dt, 51)
        c["q"] *= 4                              # scores of tens: maxima that grow for a while
        top = torch.finfo(dt).max
        c["v_cache"] = (c["v_cache"].sign() * top * (0.5 + 0.47 * torch.rand(c["v_cache"].shape))).to(dt)
        c["v_cache"][..., :5] = 0.97 * top       # (columns of equal values, clear of the largest by more than P's rounding)
        _check_attention(gpu_lib, c)
        _check_attention(gpu_lib, c, scale=0.0)


@pytest.mark.parametrize("N,D", [(1, 64), (6, 128), (40, 64)])
def test_small_values(gpu_lib, N, D):
    """Values down to 1e-20 keep their relative precision."""
    c = ref.case(2, N, 4, 2, D, 16, (300, 1500), BF, 52)
    c["q"] *= 4
    c["v_cache"] = (c["v_cache"].float() * 1e-20).to(BF)
    _check_attention(gpu_lib, c)

