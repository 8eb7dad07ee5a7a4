"""Gradients written beside the logits in one buffer: rows that share no
element are accepted and right, views shifted into the logits are refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pp():
    import __graft_entry__
    __graft_entry__.build()
    import post_processing_gb300
    return post_processing_gb300


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [100, 999, 20001])
def test_rows_between_the_logits(pp, cols, dtype):
    rows = 5
    buf = torch.randn((rows, 2 * cols + 3), device="cuda").to(dtype)
    x, out = buf[:, :cols], buf[:, cols + 1:2 * cols + 1]
    keep = buf.clone()
    tok = torch.arange(rows, device="cuda")
    f = pp.logprobs(x, tok, k=8)
    one = torch.ones(rows, device="cuda")
    want = pp.logprobs_backward(x, tok, f.stats, f.entropy, one, one)
    assert torch.equal(pp.logprobs_backward(x, tok, f.stats, f.entropy, one, one, out=out), want)
    d = pp.distill(x, f.top_idx, f.top_logprob, tail=True)
    got = pp.distill(x, f.top_idx, f.top_logprob, tail=True, out=pp.Distill(torch.empty_like(d.loss), out))
    assert torch.equal(out, d.grad) and torch.equal(got.loss, d.loss)
    keep[:, cols + 1:2 * cols + 1] = out
    assert torch.equal(buf, keep), "written outside the gradient's rows"
    for shifted in (buf[:, 1:cols + 1], buf[:, cols - 1:2 * cols - 1]):
        with pytest.raises(pp.WsError, match="overlaps"):
            pp.logprobs_backward(x, tok, f.stats, f.entropy, one, one, out=shifted)
        with pytest.raises(pp.WsError, match="overlaps"):
            pp.distill(x, f.top_idx, f.top_logprob, out=pp.Distill(torch.empty_like(d.loss), shifted))
    torch.cuda.synchronize()
    assert torch.equal(buf, keep)
