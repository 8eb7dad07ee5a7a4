"""Calls on a stream of their own, without a GPU: results come from that
stream's memory, and inputs and results are held for every stream that uses
them.  (A result from the current stream's memory could be written while work
that is still queued there reads the block under its last owner.)"""
import pytest
import torch

import fake_cuda

OWN = 0x77


@pytest.fixture
def api():
    import __graft_entry__
    __graft_entry__.build()
    from post_processing_gb300 import api
    return api


def logits_calls(api, **kw):
    T = fake_cuda.Tensor
    x, tok, per_row = T((4, 100)), T((4,), torch.int64), T((4,))
    ids, lq, stats = T((4, 5), torch.int32), T((4, 5)), T((4, 2))
    return {
        "logprobs": ((x, tok), lambda: api.logprobs(x, tok, k=3, **kw)),
        "logprobs_backward": ((x, tok, stats, per_row),
                              lambda: api.logprobs_backward(x, tok, stats, per_row, per_row, per_row, **kw)),
        "distill": ((x, ids, lq, per_row), lambda: api.distill(x, ids, lq, per_row, **kw)),
        "distill loss": ((x, ids, lq), lambda: api.distill(x, ids, lq, grad=False, **kw)),
    }


def tensors(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["logprobs", "logprobs_backward", "distill", "distill loss"])
def test_logits_results_belong_to_the_calls_stream(api, monkeypatch, name, raw):
    cuda = fake_cuda.Cuda(monkeypatch, api)
    inputs, call = logits_calls(api, stream=OWN if raw else fake_cuda.Stream(OWN))[name]
    out = call()
    assert cuda.calls[0][1][-1] == OWN
    for t in tensors(out):
        assert t.made_on == OWN
        assert 0x10 in t.held_for, "read on the current stream afterwards"
    for t in inputs:
        assert OWN in t.held_for


@pytest.mark.parametrize("name", ["logprobs", "logprobs_backward", "distill", "distill loss"])
def test_logits_calls_on_the_current_stream_hold_nothing(api, monkeypatch, name):
    cuda = fake_cuda.Cuda(monkeypatch, api)
    for stream in (None, 0x10, fake_cuda.Stream(0x10)):
        inputs, call = logits_calls(api, stream=stream)[name]
        out = call()
        assert cuda.calls[-1][1][-1] == 0x10
        for t in tensors(out) + list(inputs):
            assert not t.held_for
            assert t.made_on in (0x10, None)
