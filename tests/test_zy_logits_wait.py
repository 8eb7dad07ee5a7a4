"""A copy that does not come in time, in the log-probability kernel whose
clusters read long rows by bulk copies: the wait runs out (a short limit and a
copy that is never issued; no fault), the device error word says so, every
result of the row is written (NaN, and no index that nobody chose), and the
next call is right.  (Named to run after the tests that expect a clean word.)"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pp():
    import __graft_entry__
    __graft_entry__.build()
    import post_processing_gb300
    return post_processing_gb300


def lost(pp, x, tok, k, limit_us):
    B, (rows, cols) = pp.binding, x.shape
    dtype = {torch.float32: B.WS_DTYPE_F32, torch.float16: B.WS_DTYPE_F16, torch.bfloat16: B.WS_DTYPE_BF16}[x.dtype]
    desc = B.ws_logprobs_desc(rows, cols, x.stride(0), dtype, B.WS_INDEX_I64, k, 1.0)
    out = [torch.full((rows,), 3.0, device="cuda") for _ in range(3)] + [torch.full((rows, 2), 3.0, device="cuda")]
    top = [torch.full((rows, k), 3.0, device="cuda"), torch.full((rows, k), 2 ** 30, dtype=torch.int32, device="cuda")] if k else [None] * 2
    st = B.ws_logprobs_selftest_wait_timeout(desc, x.data_ptr(), tok.data_ptr(), *(t.data_ptr() for t in out),
                                             *(None if t is None else t.data_ptr() for t in top), limit_us,
                                             torch.cuda.current_stream().cuda_stream)
    return st, out, top


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 131072), (3, 40003), (100, 131072)])
def test_every_result_of_a_lost_row_is_written(pp, rows, cols, dtype):
    B = pp.binding
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((rows, cols), generator=g, device="cuda").to(dtype)
    tok = torch.arange(rows, device="cuda")
    for k in (0, 1, 32):
        want = pp.logprobs(x, tok, k=k)
        assert B.ws_device_error(True) == (0, 0)
        st, out, top = lost(pp, x, tok, k, 2000)
        assert st == B.WS_OK, B.ws_last_error()
        torch.cuda.synchronize()
        assert B.ws_device_error(True) == (0, 1)
        logprob, entropy, lse, stats = out
        assert logprob.isnan().all() and entropy.isnan().all() and (lse == np.inf).all()
        assert (stats[:, 0] == np.inf).all() and stats[:, 1].isnan().all()
        if k:
            assert top[0].isnan().all()
            assert (top[1][::2] == -1).all(), "even rows lose every block's run"
            assert ((top[1][1::2] >= 0) & (top[1][1::2] < cols)).all(), "odd rows the last block's"
        again = pp.logprobs(x, tok, k=k)
        assert all(torch.equal(a, b) for a, b in zip(again, want) if a is not None)
        assert B.ws_device_error(True) == (0, 0)


def test_refusals(pp):
    B = pp.binding
    x, tok = torch.zeros((2, 1000), device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    assert lost(pp, x, tok, 4, 2000)[0] == B.WS_ERR_UNSUPPORTED
    for limit in (0, 1000001):
        assert lost(pp, x, tok, 4, limit)[0] == B.WS_ERR_INVALID_ARGUMENT
    torch.cuda.synchronize()
    assert B.ws_device_error(True) == (0, 0)
