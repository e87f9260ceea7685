"""Slot weights where rows, keys or lse are not finite, over pages of which tiles differ, and in
what lies between the first tokens and a window."""
import math

import pytest
import torch

import chunk_reference as cref
from test_gpu_budget import add_weights, check_weights
from test_gpu_chunk import case
from test_gpu_target import _same
from test_gpu_waits import withheld  # noqa: F401  (a fixture)

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


@pytest.mark.parametrize("spoil", ["nan", "inf", "key"])
@pytest.mark.parametrize("N,D,ctx", [(1, 64, (300, 20)), (6, 128, (90, 700)), (32, 64, (300, 5)), (150, 128, (300, 0)),
                                     (150, 64, (0, 900))])
def test_rows_of_lse_minus_infinity_add_nothing_whatever_they_score(gpu_lib, N, D, ctx, spoil):
    """Rows that a caller takes out so: their queries are NaN, or infinite (scores of all
    signs), or every row's key is NaN somewhere."""
    c = case(2, N, 8, 2, D, 16, ctx, FP if D == 64 else BF, 9)
    out = torch.zeros((2, N, 8), dtype=torch.bool)
    out[0, N // 2] = True
    out[1, :, 5] = True
    out[1, N - 1, 1:3] = True
    q = c["q"].clone()
    if spoil == "nan":
        q[out] = math.nan
    elif spoil == "inf":
        q[out] = 0.0
        q[..., 7][out] = math.inf
    c["q"] = q
    _, lse, _, _ = cref.attention(c)
    lse = lse.float()
    lse[out] = -math.inf
    if spoil == "key":  # (other rows that see the slot spoil it, in its own place alone)
        for b in range(2):
            s = int(c["ctx_len"][b]) // 2
            c["k_cache"][c["page_table"][b, s // 16].long(), s % 16, 1, 3] = math.nan
            s = int(c["ctx_len"][b]) + N - 1
            c["k_cache"][c["page_table"][b, s // 16].long(), s % 16] = math.inf
    assert bool(torch.isfinite(lse[~out]).all())
    w = start(c)
    # (of these rows the plain form takes nothing, so any queries will do; its tolerance of
    # finite ones is theirs, 0, while one of NaN would be 0 times NaN)
    want, tol = cref.weights({**c, "q": torch.where(out[..., None], torch.zeros_like(q), q)}, lse, w, decay=0.5)
    r = add_weights(gpu_lib, c, lse, w, decay=0.5)
    _same(r["weights"], want, tol, "weights")
    lse[:] = -math.inf
    r = add_weights(gpu_lib, c, lse, w, decay=1.0)
    assert torch.equal(r["weights"].cpu(), w)


@pytest.mark.parametrize("B,N,Hq,Hkv,D,ctx,window", [
    (1, 1, 8, 2, 64, 5000, 0),      # an item in parts
    (40, 3, 8, 2, 128, 300, 0),     # items that are whole
    (2, 200, 8, 2, 64, 700, 150)])  # blocks of rows, and slots that nobody sees
def test_weights_outlive_tiles_that_do_not_arrive(gpu_lib, withheld, B, N, Hq, Hkv, D, ctx, window):  # noqa: F811
    """A call that gives up leaves every entry as it was or as it should become."""
    lib = gpu_lib
    c = case(B, N, Hq, Hkv, D, 16, ctx, BF, 73)
    _, lse, _, _ = cref.attention(c, window, 4)
    lse, w = lse.float(), start(c)
    good = add_weights(lib, c, lse, w, window=window, sinks=4, decay=0.5)
    with withheld:
        lost = add_weights(lib, c, lse, w, window=window, sinks=4, decay=0.5, ws=good["ws"])
    assert lib.get_device_error(good["ws"], clear=True) == lib.DEVERR_TIMEOUT
    got = lost["weights"].cpu()
    assert bool(((got == w) | (got == good["weights"].cpu())).all())
    again = add_weights(lib, c, lse, w, window=window, sinks=4, decay=0.5, ws=good["ws"])
    assert lib.get_device_error(good["ws"]) == 0 and torch.equal(again["weights"], good["weights"])


@pytest.mark.parametrize("page", [2, 12, 40, 72, 130, 136, 201])
def test_page_sizes(gpu_lib, page):
    """Pages whose parts make a tile, ones that need whole pages, and both kinds above 128."""
    for N, D, order in ((1, 64, "slot"), (60, 128, "slot"), (60, 128, "head"), (210, 64, "slot")):
        c = case(3, N, 8, 2, D, page, (0, 131, 620), BF, page, order=order)
        check_weights(gpu_lib, c, decay=0.5)
        check_weights(gpu_lib, c, 150, 9, decay=0.5)


@pytest.mark.parametrize("decay", [0.0, 0.5, -1.0])
@pytest.mark.parametrize("sinks", [0, 4, 300])
@pytest.mark.parametrize("page", [1, 5, 16, 201])
def test_what_no_token_sees_fades(gpu_lib, page, sinks, decay):
    """Slots between the first tokens and the window, of tiles that nobody looks at and of ones
    that somebody does."""
    for N, D in ((1, 64), (70, 128)):
        c = case(4, N, 8, 2, D, page, (99, 1500, 3001, 700), BF, 74, fill="random")
        check_weights(gpu_lib, c, 100, sinks, decay=decay)


@pytest.mark.parametrize("order", ["slot", "head"])
@pytest.mark.parametrize("page", [1, 3, 5, 12, 130, 201])
def test_odd_pages_out_of_range(gpu_lib, page, order):
    lib = gpu_lib
    for N, D in ((1, 64), (50, 128), (200, 64)):
        c = case(2, N, 8, 2, D, page, (150, 420), BF, 60 + page, fill="random", order=order)
        c["page_table"][0, 100 // page] = c["k_cache"].shape[0]
        c["page_table"][1, 300 // page] = -2
        check_weights(lib, c, decay=0.9, error=lib.DEVERR_BAD_PAGE)
        check_weights(lib, c, 330, 2, decay=0.9, error=lib.DEVERR_BAD_PAGE)
