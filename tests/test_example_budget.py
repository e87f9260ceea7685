"""The example of decoding with a budgeted cache: it runs, and a budget that nothing exceeds
changes nothing."""
import pytest
import torch

from examples.budget_decode import decode
from examples.tree_decode import Decoder

pytestmark = pytest.mark.gpu


def test_budgeted_decoding_runs(gpu_lib):
    model = Decoder(V=300, layers=2, dim=128, Hq=4, Hkv=2, D=64)
    prompt = torch.randint(0, 300, (3, 333), dtype=torch.int32, device="cuda",
                           generator=torch.Generator(device="cuda").manual_seed(1))
    whole = decode(model, prompt, 40, 1000)
    other = decode(model, prompt, 40, 400, spare=8)
    cut = decode(model, prompt, 40, 64, spare=8)
    assert torch.equal(whole["tokens"], other["tokens"]) and whole["slots"] == 373
    assert cut["slots"] == 72 and cut["tokens"].shape == (3, 40)
    for r in (whole, other, cut):
        assert not any(r["errors"].values())
