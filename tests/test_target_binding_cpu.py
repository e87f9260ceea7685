"""What the binding of the target pass's operators refuses before any pointer
reaches the library: tensors that cannot hold a result, tensors of several
devices.  Stand-ins play the CUDA tensors, and nothing is launched."""
import pytest
import torch

import target_reference as ref
import test_target_cpu as abi
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
    monkeypatch.setattr(bd, "_current_device", lambda: 0, raising=False)


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


def _append(c, **kw):
    bd.ssd_kv_append(c["q"], c["k"], c["v"], c["k_cache"], c["v_cache"], c["page_table"], c["ctx_len"],
                     parent=c["parent"], n_nodes=c["n_nodes"], cos_sin=c["cos_sin"], q_norm=c["q_norm"],
                     k_norm=c["k_norm"], ws=c["ws"], out={"q": c["out"]}, **kw)


def _attend(c, **kw):
    bd.ssd_tree_attention(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["ctx_len"], parent=c["parent"],
                          n_nodes=c["n_nodes"], ws=c["ws"], out={"out": c["out"], "lse": c["lse"]}, **kw)


def _commit(c, **kw):
    bd.ssd_kv_commit(c["k_cache"], c["v_cache"], c["page_table"], c["ctx_len"], c["accept_len"], c["out_node"],
                     ws=c["ws"], out={"ctx_len": c["new_len"]}, **kw)


def _answer(c, **kw):
    bd.ssd_logprobs(c["logits"], c["tok"], 2, c["T"], rows=c["rows"], ws=c["ws"],
                    out={k: c[k] for k in ("logprob", "entropy", "rank", "top_tok", "top_logprob")}, **kw)


def _all():
    """Every tensor of the four calls."""
    c = _case()
    c.update(n_nodes=torch.tensor([3, 2], dtype=I32), cos_sin=torch.zeros(64, 64), q_norm=torch.ones(64, dtype=BF),
             k_norm=torch.ones(64, dtype=BF), out=torch.empty((2, 3, 4, 64), dtype=BF), lse=torch.empty((2, 3, 4)),
             accept_len=torch.tensor([1, 0], dtype=I32), out_node=torch.ones((2, 3), dtype=I32),
             new_len=torch.empty(2, dtype=I32), logits=torch.zeros(6, 100), tok=torch.zeros(5, dtype=I32),
             T=torch.ones(5), rows=torch.zeros(5, dtype=I32), ws=_ws(), **_logprob_outputs())
    return {k: gpu(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}


TENSORS = {
    _append: "q k v k_cache v_cache page_table ctx_len parent n_nodes cos_sin q_norm k_norm ws out",
    _attend: "q k_cache v_cache page_table ctx_len parent n_nodes ws out lse",
    _commit: "k_cache v_cache page_table ctx_len accept_len out_node ws new_len",
    _answer: "logits tok T rows ws logprob entropy rank top_tok top_logprob"}


@needs_no_gpu
@pytest.mark.parametrize("call", TENSORS, ids=lambda f: f.__name__)
def test_tensors_of_one_device(no_launch, monkeypatch, call):
    """A call whose tensors lie on several devices, or on another than the
    current one, starts no kernel."""
    c = _all()
    with pytest.raises(Launched):
        call(c)
    for name in TENSORS[call].split():
        with pytest.raises(ValueError, match="lie"):
            call({**c, name: gpu(c[name], OnOtherGpu)})
        with pytest.raises(ValueError, match="CUDA tensor"):
            call({**c, name: torch.Tensor._make_subclass(torch.Tensor, c[name])})
    other = {k: gpu(v, OnOtherGpu) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    with pytest.raises(ValueError, match="current device"):
        call(other)
    monkeypatch.setattr(bd, "_current_device", lambda: 1)
    with pytest.raises(Launched):
        call(other)
    with pytest.raises(ValueError, match="current device"):
        call(c)


@needs_no_gpu
@pytest.mark.parametrize("call", TENSORS, ids=lambda f: f.__name__)
def test_stream_of_the_tensors_device(no_launch, call):
    class Stream:
        cuda_stream, device_index = 5, 0

    class OtherStream(Stream):
        device_index = 1
    for stream in (Stream(), 7):
        with pytest.raises(Launched):
            call(_all(), stream=stream)
    with pytest.raises(ValueError, match="stream"):
        call(_all(), stream=OtherStream())


@needs_no_gpu
@pytest.mark.parametrize("call,name", [(_append, "ctx_len"), (_attend, "ctx_len"), (_commit, "ctx_len"),
                                       (_commit, "accept_len")], ids=lambda x: getattr(x, "__name__", x))
def test_missing_lengths(no_launch, call, name):
    with pytest.raises(TypeError, match=name):
        call({**_all(), name: None})


@needs_no_gpu
@pytest.mark.parametrize("page_size,most", [(1, (1 << 31) - 258), (5, ((1 << 31) - 257) // 5 - 1),
                                            (16, ((1 << 31) - 257) // 16 - 1), (1 << 20, 2046)])
def test_tables_at_the_end_of_32_bits(lib, page_size, most):  # noqa: F811
    """Tables whose last slots, rounded up to a page or a tile of 128, would not
    be counted in 32 bits are refused; the last that fit reach CUDA (which is not
    there)."""
    def kv(width):
        return abi._kv(page_size=page_size, max_pages=width, table_stride=width)

    def commit(lib, kv):
        return lib.ssd_kv_commit(kv, 1, 0, 0, 2, 4, abi.P, abi.P, abi.P, abi.P + 64, abi.P, 256, None)
    for call in (abi._attend, abi._append, commit):
        assert call(lib, kv=kv(most + 1)) == abi.INVALID
        assert call(lib, kv=kv(most)) == 3


@needs_no_gpu
def test_batches_at_the_end_of_32_bits(lib):  # noqa: F811
    for N, most in ((1, (1 << 31) - 1025), (64, ((1 << 31) - 1025) // 64)):
        for call in (abi._attend, abi._append):
            assert call(lib, nodes=abi._nodes(B=most + 1, N=N)) == abi.INVALID
            assert call(lib, nodes=abi._nodes(B=most, N=N)) == 3


@needs_no_gpu
def test_commit_lengths_that_overlap(lib):  # noqa: F811
    """New lengths over a part of the old ones: blocks of other layers would read
    what the first has written."""
    def commit(new, ctx=abi.P, acc=abi.P + 4096, B=8):
        return lib.ssd_kv_commit(abi._kv(), 1, 0, 0, B, 4, ctx, acc, abi.P + 8192, new, abi.P, 256, None)
    for at in (abi.P, abi.P + 4096):
        for off in (-28, -4, 0, 4, 28):
            assert commit(at + off) == abi.INVALID
        assert commit(at - 32) == 3 and commit(at + 32) == 3


@needs_no_gpu
def test_scales_beyond_32_bits(lib):  # noqa: F811
    """A scale that is infinite in units of log 2."""
    for scale in (2.5e38, 3.4e38, -3.4e38):
        assert abi._attend(lib, scale=scale) == abi.INVALID
    for scale in (2e38, -1e38, 1e-40, 0.0):
        assert abi._attend(lib, scale=scale) == 3
