"""The logits calls need no workspace and allocate nothing: the device's free
memory and torch's allocation count stay over calls through the C ABI, in every
kernel, and each call is one kernel in a captured graph."""
import ctypes

import pytest
import torch

import cudart

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from post_processing_gb300 import binding
    return binding


# short rows, rows of a warp, of a block, of a cluster; past what a cluster holds (float32)
SHAPES = [(4, 500), (900, 9000), (200, 20001), (3, 131072), (2, 400001)]


def calls(B, rows, cols, k=8):
    x = torch.randn((rows, cols), device="cuda")
    tok = torch.zeros(rows, dtype=torch.int64, device="cuda")
    logprob, entropy, lse, one, loss = (torch.ones(rows, device="cuda") for _ in range(5))
    stats, top = torch.empty((rows, 2), device="cuda"), torch.empty((rows, k), device="cuda")
    idx, grad = torch.empty((rows, k), dtype=torch.int32, device="cuda"), torch.empty_like(x)
    d = B.ws_logprobs_desc(rows, cols, cols, B.WS_DTYPE_F32, B.WS_INDEX_I64, k, 1.0)
    e = B.ws_distill_desc(rows, cols, cols, cols, B.WS_DTYPE_F32, B.WS_INDEX_I32, k, B.WS_DISTILL_TAIL, 1.0)
    p = lambda t: t.data_ptr()  # noqa: E731
    held = (x, tok, logprob, entropy, lse, one, loss, stats, top, idx, grad)
    return held, [
        lambda s: B.check(B.ws_logprobs(d, p(x), p(tok), p(logprob), p(entropy), p(lse), p(stats), p(top), p(idx), s)),
        lambda s: B.check(B.ws_logprobs_backward(d, p(x), p(tok), p(stats), p(entropy), p(one), p(one), p(grad), cols, s)),
        lambda s: B.check(B.ws_distill(e, p(x), p(idx), p(top), p(one), p(loss), p(grad), s))]


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_nothing_is_allocated(B, rows, cols):
    held, run = calls(B, rows, cols)
    s = torch.cuda.current_stream().cuda_stream
    for call in run:
        call(s)                                    # the first call loads the kernels
    torch.cuda.synchronize()
    count = torch.cuda.memory_stats()["allocation.all.allocated"]
    free = torch.cuda.mem_get_info()[0]
    for _ in range(20):
        for call in run:
            call(s)
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == count


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_each_call_is_one_kernel(B, rows, cols):
    rt = cudart._cudart()
    held, run = calls(B, rows, cols)
    for call in run:
        call(torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    stream = ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(stream), 1) == 0
    try:
        for call in run:
            graph, nodes = ctypes.c_void_p(), ctypes.c_size_t(0)
            assert rt.cudaStreamBeginCapture(stream, 1) == 0   # of this thread's calls
            call(stream.value)
            assert rt.cudaStreamEndCapture(stream, ctypes.byref(graph)) == 0
            assert rt.cudaGraphGetNodes(graph, None, ctypes.byref(nodes)) == 0
            assert nodes.value == 1
            assert rt.cudaGraphDestroy(graph) == 0
    finally:
        assert rt.cudaStreamDestroy(stream) == 0
