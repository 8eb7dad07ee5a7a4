"""Tensors and streams of another device than the call's, without a second
GPU: the library launches on the current device, so they are refused before
anything is enqueued."""
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


def operands(api):
    """name -> (call, its operands by name)"""
    i32, i64 = torch.int32, torch.int64
    row = lambda: T((4,))  # noqa: E731
    lp = dict(logits=T((4, 100)), tokens=T((4,), i64), out=api.Logprobs(row(), row(), row(), T((4, 2)), T((4, 3)), T((4, 3), i32)))
    bw = dict(logits=T((4, 100)), tokens=T((4,), i64), stats=T((4, 2)), entropy=row(), grad_logprob=row(), grad_entropy=row(),
              out=T((4, 100)))
    ds = dict(logits=T((4, 100)), teacher_idx=T((4, 5), i32), teacher_logprob=T((4, 5)), weight=row(),
              out=api.Distill(row(), T((4, 100))))
    return [(lambda **kw: api.logprobs(k=3, **kw), lp), (api.logprobs_backward, bw), (api.distill, ds)]


def moved(kw, name, field=None):
    """The operands with one of them on the second device."""
    def there(t):
        return T(t.shape, t.dtype, device=1)
    if field is None:
        return {**kw, name: there(kw[name])}
    return {**kw, name: kw[name]._replace(**{field: there(getattr(kw[name], field))})}


@pytest.mark.parametrize("which", range(3))
def test_operands_of_another_device(api, monkeypatch, which):
    cuda = fake_cuda.Cuda(monkeypatch, api)
    call, kw = operands(api)[which]
    call(**kw)
    assert len(cuda.calls) == 1
    places = [(n, f) for n, v in kw.items() for f in (v._fields if isinstance(v, tuple) else (None,))]
    assert len(places) >= 6
    for name, field in places:
        with pytest.raises(ValueError, match="cuda:"):
            call(**moved(kw, name, field))
    assert len(cuda.calls) == 1, "enqueued all the same"


@pytest.mark.parametrize("which", range(3))
def test_a_device_that_is_not_the_current_one(api, monkeypatch, which):
    cuda = fake_cuda.Cuda(monkeypatch, api)
    cuda.current_device = 1
    call, kw = operands(api)[which]
    with pytest.raises(ValueError, match="current device"):
        call(**kw)
    assert not cuda.calls


def test_earlier_calls_on_a_device_that_is_not_the_current_one(api, monkeypatch):
    cuda = fake_cuda.Cuda(monkeypatch, api)
    cuda.current_device = 1
    pre, det = api.B.preprocess_desc(64, 48, 32, 32), api.B.detect_desc(in_w=320, in_h=192, reg_max=8, num_classes=3, conf=0.3)
    for call in (lambda: api.preprocess(T((2, 48, 64, 3), torch.uint8), pre), lambda: api.topk(T((4, 100)), 5),
                 lambda: api.detect(T((1, 35, 100)), det), lambda: api.topk_workspace(4, 50000, 5, "cuda:0"),
                 lambda: api.detect_workspace(det, 1, "cuda:0")):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert not cuda.calls


@pytest.mark.parametrize("which", range(3))
def test_a_stream_of_another_device(api, monkeypatch, which):
    cuda = fake_cuda.Cuda(monkeypatch, api)
    call, kw = operands(api)[which]
    with pytest.raises(ValueError, match="stream"):
        call(**kw, stream=fake_cuda.Stream(0x77, device=1))
    assert not cuda.calls
    call(**kw, stream=fake_cuda.Stream(0x77, device=0))
    assert cuda.calls[0][1][-1] == 0x77
