"""Slot weights where rows, keys or lse are not finite, over pages of which tiles differ, and in
what lies between the first tokens and a window."""
import math

import pytest
import torch

import chunk_reference as cref
from test_gpu_budget import add_weights, check_weights
from test_gpu_chunk import case
from test_gpu_target import _same

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def start(c, extra=3):
    B, H = c["q"].shape[0], c["k_cache"].shape[2]
    return torch.rand((B, H, int(c["ctx_len"].max()) + c["N"] + extra), generator=torch.Generator().manual_seed(3)) * 3


@pytest.mark.parametrize("window,sinks", [(0, 0), (25, 2)])
@pytest.mark.parametrize("N,D", [(1, 64), (20, 128), (150, 64)])
def test_nan_lse_reaches_the_slots_that_its_row_sees(gpu_lib, N, D, window, sinks):
    """exp(x - NaN) is NaN, of a slot that the row does not see nothing."""
    c = case(3, N, 8, 2, D, 16, (100, 30, 400), BF, 8)
    _, lse, _, _ = cref.attention(c, window, sinks)
    lse = lse.float()
    rows = [(0, N // 2, 1), (2, 0, 7)]
    for at in rows:
        lse[at] = -math.inf
    w = start(c)
    want, tol = cref.weights(c, lse, w, window, sinks, decay=0.5)
    for b, i, h in rows:
        L = int(c["ctx_len"][b])
        see = cref.seen(L, N, window, sinks)[i]
        want[b, h // 4, :L + N][see] = math.nan
        lse[b, i, h] = math.nan
    r = add_weights(gpu_lib, c, lse, w, window=window, sinks=sinks, decay=0.5)
    _same(r["weights"], want, tol, "weights")
    assert gpu_lib.get_device_error(r["ws"]) == 0
