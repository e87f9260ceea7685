"""Page ids of slots that no token sees: a cache may have given those pages back."""
import pytest
import torch

import chunk_reference as cref
from test_gpu_budget import add_weights
from test_gpu_chunk import case, check
from test_gpu_target import _same

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
PAGES = [1, 2, 3, 5, 16, 48, 128, 130, 201]


def seen_pages(c, window, sinks):
    """[B, width] truth values: pages with a slot that some token sees."""
    B, width = c["page_table"].shape
    see = torch.zeros((B, width), dtype=torch.bool)
    for b in range(B):
        s = cref.seen(int(c["ctx_len"][b]), c["N"], window, sinks).any(0).nonzero()[:, 0]
        see[b, s // c["page"]] = True
    return see


def sums(lib, c, window, sinks, error):
    _, lse, _, _ = cref.attention(c, window, sinks)
    lse = lse.float()
    w = torch.rand((c["q"].shape[0], 2, int(c["ctx_len"].max()) + c["N"]), generator=torch.Generator().manual_seed(4))
    want, tol = cref.weights(c, lse, w, window, sinks, decay=0.5)
    r = add_weights(lib, c, lse, w, window=window, sinks=sinks, decay=0.5)
    assert lib.get_device_error(r["ws"]) == error
    _same(r["weights"], want, tol, "weights")


def spoilt(N, D, page, dt, window, sinks, ctx=(900, 333, 1301)):
    """A case whose pages that nobody sees have ids of no page, of both kinds."""
    c = case(3, N, 8, 2, D, page, ctx, dt, 90 + page, fill="random")
    gone = ~seen_pages(c, window, sinks)
    assert bool(gone.any())
    c["page_table"][gone] = -1
    c["page_table"][:, ::2][gone[:, ::2]] = c["k_cache"].shape[0] + 7
    return c


@pytest.mark.parametrize("window,sinks", [(100, 4), (130, 0), (37, 129)])
@pytest.mark.parametrize("page", PAGES)
def test_pages_given_back_are_no_error(gpu_lib, page, window, sinks):
    for N, D, dt in ((1, 64, BF), (9, 128, FP), (140, 64, BF)):
        c = spoilt(N, D, page, dt, window, sinks)
        check(gpu_lib, c, window, sinks)
        sums(gpu_lib, c, window, sinks, 0)


@pytest.mark.parametrize("page", PAGES)
def test_the_first_and_last_seen_slots_still_count(gpu_lib, page):
    """The same with one more id out of range, of a page that holds a seen slot."""
    lib = gpu_lib
    window, sinks = 100, 5
    for N, D, dt in ((1, 64, BF), (9, 128, FP), (140, 64, BF)):
        for slot in (0, sinks - 1, 333 - window + 1, 333 + N - 1):
            c = spoilt(N, D, page, dt, window, sinks)
            c["page_table"][1, slot // page] = -5
            check(lib, c, window, sinks, error=lib.DEVERR_BAD_PAGE)
            sums(lib, c, window, sinks, lib.DEVERR_BAD_PAGE)
