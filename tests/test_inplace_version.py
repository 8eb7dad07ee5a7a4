"""Gradients written over the logits count up autograd's version of them: a
graph that saved the logits then raises an error where it would otherwise use
gradients in their place.  Without a GPU by stand-ins; on one with a graph."""
import pytest
import torch

import fake_cuda

T = fake_cuda.Tensor


@pytest.fixture
def api():
    import __graft_entry__
    __graft_entry__.build()
    from post_processing_gb300 import api
    return api


@pytest.fixture
def bumped(api, monkeypatch):
    fake_cuda.Cuda(monkeypatch, api)
    seen = []
    monkeypatch.setattr(torch.autograd.graph, "increment_version", seen.append)
    return seen


def test_in_place(api, bumped):
    x, row = T((4, 100)), T((4,))
    tok, stats, ids, lq = T((4,), torch.int64), T((4, 2)), T((4, 5), torch.int32), T((4, 5))
    api.logprobs_backward(x, tok, stats, row, row, out=x)
    assert bumped == [x]
    api.distill(x, ids, lq, out=api.Distill(row, x))
    assert bumped == [x, x]
    view = T((4, 100))   # another tensor of the same memory
    api.logprobs_backward(x, tok, stats, row, row, out=view)
    assert bumped == [x, x, view]


def test_elsewhere(api, bumped):
    x, row, out = T((4, 100)), T((4,)), T((4, 100), address=1 << 21)
    tok, stats, ids, lq = T((4,), torch.int64), T((4, 2)), T((4, 5), torch.int32), T((4, 5))
    for o in (None, out):
        api.logprobs_backward(x, tok, stats, row, row, out=o)
        api.distill(x, ids, lq, out=None if o is None else api.Distill(row, o))
    api.distill(x, ids, lq, grad=False)
    assert not bumped


def test_a_refused_call_changes_nothing(api, bumped, monkeypatch):
    x, row = T((4, 100)), T((4,))
    monkeypatch.setattr(api.B, "ws_logprobs_backward", lambda *a: 1)
    with pytest.raises(api.B.WsError):
        api.logprobs_backward(x, T((4,), torch.int64), T((4, 2)), row, row, out=x)
    assert not bumped


@pytest.mark.gpu
def test_a_graph_that_saved_the_logits(api):
    import post_processing_gb300 as pp
    w = torch.randn((16, 500), device="cuda", requires_grad=True)
    for call in ("backward", "distill"):
        hidden = torch.randn((4, 16), device="cuda")
        logits = hidden @ w
        saved = (logits * logits).sum()          # its backward pass needs the logits
        x = logits.detach()
        f = pp.logprobs(x, torch.arange(4, device="cuda"), k=5)
        if call == "backward":
            pp.logprobs_backward(x, torch.arange(4, device="cuda"), f.stats, None, f.logprob, out=x)
        else:
            pp.distill(x, f.top_idx, f.top_logprob, out=pp.Distill(f.lse, x))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.backward()
        # logits that nothing saved: their gradient goes on through what made them, here written over them
        logits = hidden @ w
        x = logits.detach()
        d = pp.distill(x, f.top_idx, f.top_logprob, out=pp.Distill(f.lse, x))
        w.grad = None
        logits.backward(d.grad.clone())
        assert torch.allclose(w.grad, hidden.t() @ d.grad, rtol=1e-3, atol=1e-5)
