"""What the binding of the target pass's operators refuses before any pointer
reaches the library: tensors that cannot hold a result, tensors of several
devices.  Stand-ins play the CUDA tensors, and nothing is launched."""
import pytest
import torch

import target_reference as ref
from speculative_decoding_verification_70_gb300 import _binding as bd
from test_abi_cpu import lib, needs_no_gpu  # noqa: F401

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class OnGpu(torch.Tensor):
    """A CPU tensor that says it lies on a GPU."""
    where = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.where


class OnOtherGpu(OnGpu):
    where = 1


def gpu(t, kind=OnGpu):
    return torch.Tensor._make_subclass(kind, t)


def _case():
    c = ref.case(2, 3, 4, 2, 64, 16, (5, 20), BF, 1)
    return {k: gpu(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def _ws(n=1 << 22):
    return gpu(torch.zeros(n, dtype=torch.uint8))


class Launched(Exception):
    pass


@pytest.fixture
def no_launch(lib, monkeypatch):  # noqa: F811
    """The library with entry points that say they were reached."""
    class Fake:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return getattr(lib, name)

            def call(*a):
                raise Launched(name)
            return call
    monkeypatch.setattr(bd, "load_library", lambda: Fake())
    monkeypatch.setattr(bd, "_raw_stream", lambda d: 0)


def _logprobs(out, K=2, R=5):
    bd.ssd_logprobs(gpu(torch.zeros(R, 100)), gpu(torch.zeros(R, dtype=I32)), K, ws=_ws(), out=out)


def _logprob_outputs(R=5, K=2, **kw):
    out = {"logprob": torch.empty(R), "entropy": torch.empty(R), "rank": torch.empty(R, dtype=I32),
           "top_tok": torch.empty((R, K), dtype=I32), "top_logprob": torch.empty((R, K))}
    out.update(kw)
    return {k: gpu(v) for k, v in out.items() if v is not None}


BAD_LOGPROB_OUT = [
    dict(logprob=torch.empty(4)), dict(logprob=torch.empty(5, dtype=torch.float64)), dict(entropy=torch.empty(4)),
    dict(entropy=torch.empty(5, dtype=BF)), dict(rank=torch.empty(3, dtype=I32)),
    dict(rank=torch.empty(5, dtype=torch.int64)), dict(top_tok=torch.empty((5, 1), dtype=I32)),
    dict(top_tok=torch.empty((5, 2), dtype=torch.int64)), dict(top_logprob=torch.empty((5, 1))),
    dict(top_logprob=torch.empty((4, 2))), dict(top_logprob=torch.empty((5, 2), dtype=BF)),
    dict(top_logprob=torch.empty((2, 5)).t()), dict(entropy=torch.empty(10)[::2])]


@needs_no_gpu
@pytest.mark.parametrize("kw", BAD_LOGPROB_OUT, ids=lambda d: "-".join("%s%s" % (k, list(v.shape)) for k, v in d.items()))
def test_logprob_outputs_of_other_sizes_and_types(no_launch, kw):
    with pytest.raises(ValueError):
        _logprobs(_logprob_outputs(**kw))


@needs_no_gpu
def test_logprob_outputs_that_fit(no_launch, monkeypatch):
    for out in (_logprob_outputs(), _logprob_outputs(logprob=torch.empty((1, 5)))):
        with pytest.raises(Launched):
            _logprobs(out)
    # the best of an earlier call are not returned as this call's
    out = _logprob_outputs()
    with pytest.raises(Launched):
        _logprobs(out, K=0)
    assert sorted(out) == ["entropy", "logprob", "rank"]
    # what is missing is made
    logits, tok, ws = gpu(torch.zeros(5, 100)), gpu(torch.zeros(5, dtype=I32)), _ws()
    made, out = [], _logprob_outputs(entropy=None, top_logprob=None)
    monkeypatch.setattr(bd.torch, "empty",
                        lambda shape, dtype, device: made.append(shape) or gpu(torch.zeros(shape, dtype=dtype)))
    with pytest.raises(Launched):
        bd.ssd_logprobs(logits, tok, 2, ws=ws, out=out)
    assert made == [(5,), (5, 2)]


@needs_no_gpu
def test_attention_and_append_outputs(no_launch):
    c = _case()
    at = (c["k_cache"], c["v_cache"], c["page_table"], c["ctx_len"])
    good = {"out": torch.empty((2, 3, 4, 64), dtype=BF), "lse": torch.empty((2, 3, 4))}
    for kw in (dict(out=torch.empty((2, 3, 4, 64))), dict(out=torch.empty((2, 3, 2, 64), dtype=BF)),
               dict(lse=torch.empty((2, 3, 2))), dict(lse=torch.empty((2, 3, 4), dtype=BF))):
        with pytest.raises(ValueError):
            bd.ssd_tree_attention(c["q"], *at, ws=_ws(), out={k: gpu(v) for k, v in {**good, **kw}.items()})
    with pytest.raises(Launched):
        bd.ssd_tree_attention(c["q"], *at, ws=_ws(), out={k: gpu(v) for k, v in good.items()})
    for q in (torch.empty((2, 3, 4, 64)), torch.empty((2, 3, 4, 32), dtype=BF)):
        with pytest.raises(ValueError):
            bd.ssd_kv_append(c["q"], c["k"], c["v"], *at, ws=_ws(), out={"q": gpu(q)})
    with pytest.raises(Launched):
        bd.ssd_kv_append(c["q"], c["k"], c["v"], *at, ws=_ws(), out={"q": gpu(good["out"])})
