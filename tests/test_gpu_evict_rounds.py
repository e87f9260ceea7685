"""Moves of few heads: a cluster takes a head's rows in rounds, the places of the next round
found by some of a CTA's threads and read by all."""
import pytest
import torch

import chunk_reference as cref
from test_gpu_budget import check_evict, evict_case

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("layers,Hkv,D,page,ctx,budget,dt", [
    (1, 1, 64, 16, 6400, 6300, BF),    # four rounds of a cluster of 8, almost nothing cut
    (1, 2, 128, 5, 7000, 4100, FP),    # five rounds, rows from far behind
    (2, 16, 128, 16, 900, 700, BF),    # clusters of four, two rounds
    (1, 64, 64, 64, 1100, 1000, FP),   # 64 heads: pairs, two rounds
    (1, 76, 64, 32, 1100, 1000, BF)])  # 76: the last number of heads with clusters
def test_every_round_takes_its_own_places(gpu_lib, layers, Hkv, D, page, ctx, budget, dt):
    """The plain form's rows, and the same again at every repeat with the pages in another
    order (so that no address of a call before is right)."""
    lib = gpu_lib
    c, w = evict_case(layers, 1, Hkv, D, page, ctx, dt, 80 + Hkv)
    check_evict(lib, c, w, budget, 3, 40, in_place=True)
    _, _, _, kept, _ = cref.evict({**c, "k_cache": c["k_cache"][:, :, :, :, :0], "v_cache": c["v_cache"][:, :, :, :, :0]},
                                  w, budget, 3, 40)
    pages = c["k_cache"].shape[1]
    kv = [c[n].cuda() for n in ("k_cache", "v_cache")]
    wg, ctx_len = w.cuda(), c["ctx_len"].cuda()
    src = kept[:, 0].long().cuda()                                # [layers, Hkv, budget]
    lyr = torch.arange(layers, device="cuda")[:, None, None].expand_as(src)
    head = torch.arange(Hkv, device="cuda")[None, :, None].expand_as(src)
    to = torch.arange(budget, device="cuda").expand_as(src)
    gen = torch.Generator().manual_seed(81)
    for _ in range(10):
        order = torch.randperm(pages, generator=gen)
        table = order[:c["page_table"].shape[1]].to(torch.int32).view(1, -1).cuda()
        page_of = table[0].long()
        want = [t.clone() for t in kv]
        for t, x in zip(want, kv):
            t[lyr, page_of[to // page], to % page, head] = x[lyr, page_of[src // page], src % page, head]
        got = [t.clone() for t in kv]
        r = lib.ssd_kv_evict(*got, table, ctx_len, wg, budget, sinks=3, recent=40)
        assert torch.equal(r["kept"][:, 0].long(), src)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert lib.get_device_error(r["ws"]) == 0
