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


def earlier_calls(api, **kw):
    T = fake_cuda.Tensor
    frames, x, head = T((2, 48, 64, 3), torch.uint8), T((4, 50000)), T((1, 35, 100))
    pre, det = api.B.preprocess_desc(64, 48, 32, 32), api.B.detect_desc(in_w=320, in_h=192, reg_max=8, num_classes=3, conf=0.3)
    return {
        "preprocess": ((frames,), lambda: api.preprocess(frames, pre, **kw)),
        "topk": ((x,), lambda: api.topk(x, 5, **kw)),
        "topk_workspace": ((), lambda: api.topk_workspace(4, 50000, 5, **kw)),
        "detect": ((head,), lambda: api.detect(head, det, **kw)),
        "detect_workspace": ((), lambda: api.detect_workspace(det, 1, **kw)),
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["preprocess", "topk", "topk_workspace", "detect", "detect_workspace"])
def test_earlier_results_and_workspaces_belong_to_the_calls_stream(api, monkeypatch, name, raw):
    """The workspace that a call makes for itself is freed when it returns, before its kernels have run: it has to be the
    stream's own memory."""
    cuda = fake_cuda.Cuda(monkeypatch, api)
    inputs, call = earlier_calls(api, stream=OWN if raw else fake_cuda.Stream(OWN))[name]
    call()
    assert {args[-1] for _, args in cuda.calls} == {OWN}
    assert cuda.made
    for t in cuda.made:
        assert t.made_on == OWN
        assert 0x10 in t.held_for
    for t in inputs:
        assert OWN in t.held_for


@pytest.mark.parametrize("name", ["preprocess", "topk", "topk_workspace", "detect", "detect_workspace"])
def test_earlier_calls_on_the_current_stream_hold_nothing(api, monkeypatch, name):
    cuda = fake_cuda.Cuda(monkeypatch, api)
    inputs, call = earlier_calls(api)[name]
    call()
    assert {args[-1] for _, args in cuda.calls} == {0x10}
    for t in cuda.made + list(inputs):
        assert not t.held_for and t.made_on in (0x10, None)


@pytest.mark.parametrize("name", ["topk", "detect"])
def test_a_given_workspace_is_held_too(api, monkeypatch, name):
    fake_cuda.Cuda(monkeypatch, api)
    ws = fake_cuda.Tensor((1000,), torch.uint8)
    earlier_calls(api, stream=OWN, workspace=ws)[name][1]()
    assert OWN in ws.held_for
