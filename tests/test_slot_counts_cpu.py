"""Numbers of slots that the library's 32 bits do not hold: cut to them they would mean another
window, other first tokens or another budget.  Nothing is launched."""
import pytest
import torch

from speculative_decoding_verification_70_gb300 import _binding as bd
from test_abi_cpu import lib, needs_no_gpu  # noqa: F401
from test_chunk_cpu import _case
from test_target_binding_cpu import Launched, _ws, gpu, no_launch  # noqa: F401

OVER = [1 << 31, 1 << 32, (1 << 32) + 7, -(1 << 32) + 7]


def calls(c, **kw):
    w, ws = gpu(torch.zeros(2, 2, 50)), _ws()
    out = {"out": gpu(torch.empty((2, c["N"], 4, 64), dtype=torch.bfloat16)), "lse": gpu(torch.empty((2, c["N"], 4)))}
    at = (c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["ctx_len"])
    if "window" in kw or "sinks" in kw:
        yield lambda: bd.ssd_chunk_attention(*at, ws=ws, out=out, **kw)
        yield lambda: bd.ssd_kv_weights(at[0], at[1], *at[3:], gpu(torch.zeros(2, c["N"], 4)), w, ws=ws, **kw)
    if "window" not in kw:
        yield lambda: bd.ssd_kv_evict(*at[1:], w, kw.get("budget", 7), ws=ws,
                                      out={"ctx_len": gpu(torch.empty(2, dtype=torch.int32)), "weights": w,
                                           "kept": gpu(torch.empty((2, 2, 7), dtype=torch.int32))},
                                      **{k: v for k, v in kw.items() if k != "budget"})


@needs_no_gpu
@pytest.mark.parametrize("name", ["window", "sinks", "recent", "budget"])
def test_counts_beyond_32_bits_are_refused(no_launch, name):  # noqa: F811
    for x in OVER:
        for call in calls(_case(), **{name: x}):
            with pytest.raises(ValueError):
                call()


@needs_no_gpu
@pytest.mark.parametrize("name", ["window", "sinks"])
def test_the_largest_counts_reach_the_library(no_launch, name):  # noqa: F811
    for call in calls(_case(), **{name: (1 << 31) - 1}):
        with pytest.raises(Launched):
            call()
