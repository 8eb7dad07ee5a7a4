"""Calls on a stream of their own while the current stream is still busy: a
block that was freed there, but that queued work still reads, must not become
the memory of a result."""
import pytest
import torch

pytestmark = pytest.mark.gpu
SPIN = 200_000_000   # clocks that the current stream is busy for: about 0.1 s


@pytest.fixture(scope="module")
def pp():
    import __graft_entry__
    __graft_entry__.build()
    import post_processing_gb300
    return post_processing_gb300


def check(elems, dtype, call):
    """call(stream) makes a result of `elems` elements while the current stream has yet to read a freed block of that size."""
    s = torch.cuda.Stream()
    call(s)                                       # warm: the library's own first-call work
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.full((elems,), 7.0, dtype=dtype, device="cuda")
    kept = torch.empty_like(block)
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    kept.copy_(block)
    del block
    got = call(s)
    s.synchronize()
    assert not torch.cuda.current_stream().query(), "the current stream was not busy while the call ran"
    torch.cuda.synchronize()
    assert (kept == 7.0).all(), "the result was written into memory that the current stream still read"
    return got


def test_logits_calls(pp):
    rows, cols = 65536, 64
    x = torch.randn((rows, cols), device="cuda").bfloat16()
    tok = torch.zeros(rows, dtype=torch.int64, device="cuda")
    f = pp.logprobs(x, tok, k=4)
    one = torch.ones(rows, device="cuda")
    torch.cuda.synchronize()
    got = check(rows * 9, torch.float32, lambda s: pp.logprobs(x, tok, k=4, stream=s))
    assert all(torch.equal(a, b) for a, b in zip(got, f))
    g = check(rows * cols, torch.bfloat16, lambda s: pp.logprobs_backward(x, tok, f.stats, f.entropy, one, one, stream=s))
    assert torch.equal(g, pp.logprobs_backward(x, tok, f.stats, f.entropy, one, one))
    d = check(rows * cols, torch.bfloat16, lambda s: pp.distill(x, f.top_idx, f.top_logprob, tail=True, stream=s))
    want = pp.distill(x, f.top_idx, f.top_logprob, tail=True)
    assert torch.equal(d.grad, want.grad) and torch.equal(d.loss, want.loss)


def test_a_result_freed_early_is_held_for_its_readers(pp):
    """A result of another stream that the current stream reads, freed before that has run, is not given to the next call."""
    rows, cols = 65536, 64
    x = torch.randn((rows, cols), device="cuda").bfloat16()
    tok = torch.zeros(rows, dtype=torch.int64, device="cuda")
    f = pp.logprobs(x, tok)
    one, s = torch.ones(rows, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    first = pp.logprobs_backward(x, tok, f.stats, None, one, stream=s)
    s.synchronize()
    want = first.clone()
    kept = torch.empty_like(first)
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    kept.copy_(first)
    del first
    pp.logprobs_backward(x, tok, f.stats, None, -one, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_topk(pp):
    rows, cols, k = 64, 200000, 32
    x = torch.randn((rows, cols), device="cuda")
    val, idx = pp.topk(x, k)
    torch.cuda.synchronize()
    assert pp.topk_workspace(rows, cols, k) is not None
    for elems in (rows * k, rows * cols // 16):
        v, i = check(elems, torch.float32, lambda s: pp.topk(x, k, stream=s))
        assert torch.equal(v, val) and torch.equal(i, idx)


def test_preprocess(pp):
    B = pp.binding
    desc = B.preprocess_desc(640, 480, 224, 224)
    frames = torch.randint(0, 256, (8, 480, 640, 3), dtype=torch.uint8, device="cuda")
    want = pp.preprocess(frames, desc)
    torch.cuda.synchronize()
    assert torch.equal(check(8 * 3 * 224 * 224, torch.float32, lambda s: pp.preprocess(frames, desc, stream=s)), want)
