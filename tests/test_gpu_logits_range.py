"""Entries near both ends of float32's range: their difference passes it, the
difference over the temperature does not."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
END = 3.0e38


@pytest.fixture(scope="module")
def pp():
    import __graft_entry__
    __graft_entry__.build()
    import post_processing_gb300
    return post_processing_gb300


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [8, 1000, 20001, 300001])
@pytest.mark.parametrize("temperature", [4.0, 1000.0, 2.0 ** 20])
def test_finite_log_probabilities_and_losses(pp, temperature, cols, dtype):
    x = torch.full((2, cols), -np.inf, device="cuda")
    x[:, 1], x[:, cols // 2], x[0, cols - 1] = END, -END, -END / 2
    x = x.to(dtype)
    v = x.double()
    # one entry holds everything, so ln p of the others is their distance; 3 roundings of it
    want = (v - v[:, 1:2]) / temperature
    tok = torch.tensor([cols // 2, cols // 2], device="cuda")
    f = pp.logprobs(x, tok, k=3, temperature=temperature)
    close = lambda a, b: torch.allclose(a.double(), b, rtol=4 * 2.0 ** -24, atol=0.0)  # noqa: E731
    assert want.gather(1, tok[:, None]).isfinite().all()
    assert close(f.logprob, want.gather(1, tok[:, None]).squeeze(1))
    assert close(f.top_logprob, want.gather(1, f.top_idx.long()))
    assert torch.equal(f.top_idx[0].cpu(), torch.tensor([1, cols - 1, cols // 2], dtype=torch.int32))
    # a teacher that holds 3/4 of its mass on the far entry; the tail class lies on the likely one, or on the third
    for ids, lq in (([cols // 2], [0.75]), ([1, cols // 2], [0.5, 0.25])):
        q = torch.tensor([lq], device="cuda").float()
        ids = torch.tensor([ids], device="cuda")
        got = pp.distill(x[:1], ids, q.log(), temperature=temperature, tail=True)
        far = want[0, cols // 2].item() * lq[-1]
        if len(lq) == 2:
            far += 0.25 * want[0, cols - 1].item()
        assert torch.allclose(got.loss.double().cpu(), torch.tensor([-far]).double(), rtol=1e-6)
        assert got.grad.isfinite().all()


@pytest.mark.parametrize("cols", [100, 9000, 300001])
def test_gradients_at_masked_tokens_and_columns(pp, cols):
    """A masked entry has no gradient but what the formulas add at a token or a teacher's column."""
    T = 0.5
    x = torch.randn((2, cols), device="cuda")
    x[0, 3], x[0, 7], x[1] = -np.inf, -np.inf, -np.inf
    tok, g = torch.tensor([3, 3], device="cuda"), torch.tensor([2.0, 2.0], device="cuda")
    f = pp.logprobs(x, tok, temperature=T)
    grad = pp.logprobs_backward(x, tok, f.stats, f.entropy, g, g, temperature=T)
    assert f.logprob[0] == -np.inf and grad[0, 3] == 2.0 / T and grad[0, 7] == 0.0
    assert not grad[1].any()
    q = torch.tensor([[0.5, 0.25]], device="cuda").repeat(2, 1)
    w = torch.tensor([3.0, 3.0], device="cuda")
    d = pp.distill(x, torch.tensor([[3, 5], [3, 5]], device="cuda"), q.log(), w, temperature=T, tail=True)
    assert d.loss[0] == np.inf and d.loss[1] == 0.0
    assert torch.allclose(d.grad[0, 3], torch.tensor(-3.0 * 0.5 / T, device="cuda"), rtol=1e-6) and d.grad[0, 7] == 0.0
    assert not d.grad[1].any()


def test_a_log_sum_exp_past_float32s_range(pp):
    """Infinite by itself; what is relative to the maximum is not."""
    x = torch.full((1, 300), END, device="cuda")
    f = pp.logprobs(x, torch.tensor([5], device="cuda"), k=2, temperature=0.5)
    assert f.lse.item() == np.inf and f.stats[0, 0] == x[0, 0]
    for v in (f.logprob, f.top_logprob, -f.entropy, -f.stats[:, 1]):
        assert torch.allclose(v, torch.full_like(v, -np.log(300.0)), rtol=1e-6)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("temperature", [2.0 ** -20, 0.0625, 17.0, 2.0 ** 20])
def test_gradients_over_the_accepted_temperatures(pp, temperature, dtype):
    """With logits of a fixed size, with ones that go by the temperature, and with a mask of the type's lowest value; the
    bounds of test_gpu_logits.py."""
    import test_gpu_logits as base
    g = np.random.default_rng(11)
    for cols in (100, 5003, 40003):
        for scale in (2.0, 4.0 * temperature):
            y = np.clip(g.normal(0.0, scale, (4, cols)), -6e4, 6e4)
            y[3, cols // 2:] = base.LOWEST[dtype]
            x, xd = base.placed(y, dtype)
            tokens = np.array([cols // 3, 0, -1, cols - 1])
            # gradients that leave float16's range by themselves are not compared: scaled to it
            a = (g.normal(0, 1, 4) * min(temperature, 1.0)).astype(np.float32)
            base.check_backward(pp, x, xd, dtype, tokens, a, (a * 0.1).astype(np.float32), temperature)
