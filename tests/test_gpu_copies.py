"""Single tokens and short chains of heads of 64, whose rows lie in the row tile two or four
times: values that are not finite, in items that are whole and in ones that are cut."""
import math

import pytest
import torch

import chunk_reference as cref
import target_reference as ref
from test_gpu_chunk import attend, case, check
from test_gpu_waits import withheld  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16

SHAPES = [
    # B, ctx: one sequence in parts, a few, more items than CTAs
    (1, (3000,)),
    (3, (40, 700, 133)),
    (90, tuple((i * 53) % 400 for i in range(90)))]


def put(c, b, slot, name, value, head=slice(None), entry=slice(None)):
    p, o = ref.where(c, b, slot)
    c[name][p, o, head, entry] = value


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("N", [1, 6, 16])
@pytest.mark.parametrize("B,ctx", SHAPES)
@pytest.mark.parametrize("dt", [BF, FP])
def test_values_that_are_not_finite(gpu_lib, B, ctx, N, window, dt):
    """NaN and infinities in slots that all rows see, that some see and that no row sees spoil
    the entries of the rows that see them, and nothing else."""
    c = case(B, N, 8, 2, 64, 16, ctx, dt, 70 + N)
    for b in range(0, B, 2):
        L = int(c["ctx_len"][b])
        put(c, b, L + N // 2, "v_cache", math.inf, entry=3)
        put(c, b, L + N // 2, "v_cache", -math.inf, entry=9)
        put(c, b, L + N - 1, "v_cache", math.nan, head=1, entry=40)
        if L > 60:
            put(c, b, L - 1, "v_cache", math.inf, head=0, entry=slice(60, 64))
            put(c, b, L - 9, "v_cache", -math.inf, head=0, entry=63)   # with the one before: NaN
            put(c, b, L // 2, "v_cache", math.nan, head=1, entry=17)   # (beyond the window)
            put(c, b, 1, "v_cache", -math.inf, head=1, entry=18)
        if b % 4 == 0:
            put(c, b, L, "k_cache", math.nan, head=1)
    check(gpu_lib, c, window, 2 if window else 0)


@pytest.mark.parametrize("G,N", [(1, 1), (8, 1), (16, 4), (5, 9)])
def test_a_row_of_nan_stays_alone(gpu_lib, G, N):
    """One query of NaN: its rows are NaN, all others have the bits that they have without it."""
    for B, ctx in SHAPES:
        c = case(B, N, 2 * G, 2, 64, 16, ctx, BF, 71)
        want = attend(gpu_lib, c)
        q = c["q"].clone()
        q[B // 2, N // 2, G] = math.nan
        got = attend(gpu_lib, {**c, "q": q})
        other = torch.ones(q.shape[:3], dtype=torch.bool)
        other[B // 2, N // 2, G] = False
        for key in ("out", "lse"):
            a, b = got[key].cpu(), want[key].cpu()
            assert torch.equal(a[other], b[other]) and bool(torch.isnan(a[~other]).all())
        assert gpu_lib.get_device_error(got["ws"]) == 0


def _us(lib, g):
    """The shortest of five calls, in microseconds."""
    r, best = None, math.inf
    for _ in range(6):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        r = lib.ssd_chunk_attention(g["q"], g["k_cache"], g["v_cache"], g["page_table"], g["ctx_len"],
                                    ws=None if r is None else r["ws"], out=r)
        b.record()
        b.synchronize()
        best = min(best, 1000 * a.elapsed_time(b))
    return best


def test_what_is_not_finite_does_not_hold_up_a_batch(gpu_lib):
    """64 sequences, one of them spoilt: a NaN query or key costs no walk over the slots (three
    times the time at most; one thread that walked alone took over a hundred times), an infinite
    value one that all threads share."""
    c = case(64, 1, 32, 8, 64, 16, 4000, BF, 72, fill="random")
    g = ref.to_gpu(c)
    plain = _us(gpu_lib, g)
    q = g["q"].clone()
    q[31] = math.nan
    assert _us(gpu_lib, {**g, "q": q}) < 3 * plain + 20
    p, o = ref.where(c, 17, 2001)
    k = g["k_cache"].clone()
    k[p, o] = math.nan
    assert _us(gpu_lib, {**g, "k_cache": k}) < 3 * plain + 20
    v = g["v_cache"].clone()
    v[p, o] = math.inf
    assert _us(gpu_lib, {**g, "v_cache": v}) < 10 * plain + 20


@pytest.mark.parametrize("B,N,Hq,Hkv,ctx", [
    (2, 8, 16, 2, 5000),    # 64 rows, two copies, items in parts
    (3, 5, 18, 2, 40),      # 45 rows, whole items
    (1, 4, 16, 2, 3000)])   # 32 rows, four copies
def test_copies_of_tiles_that_do_not_arrive(gpu_lib, withheld, B, N, Hq, Hkv, ctx):  # noqa: F811
    """The call ends with the error bit; then the same call is right, with its workspace."""
    lib = gpu_lib
    c = case(B, N, Hq, Hkv, 64, 16, ctx, BF, 75)
    good = check(lib, c)
    with withheld:
        attend(lib, c, ws=good["ws"])
    assert lib.get_device_error(good["ws"], clear=True) == lib.DEVERR_TIMEOUT
    again = attend(lib, c, ws=good["ws"])
    assert lib.get_device_error(good["ws"]) == 0
    assert torch.equal(again["out"], good["out"]) and torch.equal(again["lse"], good["lse"])
