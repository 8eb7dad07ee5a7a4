"""Distillation with the tail class where the student disagrees strongly with
its teacher: its mass off the teacher's columns is far below float32's range
(or nearly all there is), at the temperatures that are accepted.  The loss
and the gradient stay what the formulas give; they are compared with 64-bit
definitions that hold the masses as logarithms.

Bounds, in u = 2^-24 (logits_ref.py has the rest): of an entry j off the
teacher's columns the gradient is w / T (on p_j - rest c_j), with c_j its
share of the mass off them.  p_j and c_j are products of two exponentials, of
3 u a nat of their arguments and 4 u each, over a sum that is off by delta;
rest = 1 - sum q is off by eps = (2 k + 8) u, absolutely.  The loss adds rest
(ln rest - ln p_off): eps per nat of it and delta, which counts once, not
times rest, where it is taken from the difference of the masses on the
entries.
"""
import numpy as np
import pytest
import torch

import logits_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = ref.U


@pytest.fixture(scope="module")
def pp():
    import __graft_entry__
    __graft_entry__.build()
    import post_processing_gb300
    return post_processing_gb300


def lse(z):
    m = z.max(-1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(divide="ignore"):
        return m + np.log(np.exp(z - m).sum(-1, keepdims=True))


def want(x, ids, lq, w, T):
    """(loss, gradient, bound of the loss, bound of the gradient before its rounding); tail class."""
    T = float(np.float32(T))   # as the call takes it
    rows, cols = x.shape
    k, d = ids.shape[1], ref.delta(cols, cols // 256 + 32)
    eps = (2 * k + 8) * U
    z = x / T
    lp = z - lse(z)
    l = lq.astype(np.float64)
    q = np.exp(l)
    rest = 1.0 - q.sum(-1, keepdims=True)
    rest = np.where(rest < ref.TAIL_MIN, 0.0, rest)
    whole = q.sum(-1, keepdims=True) + rest
    off = np.ones((rows, cols), bool)
    np.put_along_axis(off, ids, False, -1)
    l_off = lse(np.where(off, lp, -np.inf))
    on_lp = np.take_along_axis(lp, ids, -1)
    span = np.abs(np.where(np.isfinite(lp), lp, 0.0)) + np.log(cols)
    with np.errstate(divide="ignore", invalid="ignore"):
        gap = np.where(rest > 0, np.log(rest) - l_off, 0.0)
        share = np.exp(np.where(off, lp - l_off, -np.inf))
    p = np.exp(lp)
    loss = (q * (l - on_lp)).sum(-1, keepdims=True) + rest * gap
    loss_tol = (q * (d + 4 * U * (np.abs(on_lp) + np.log(cols) + np.abs(l) + 1.0)) + (k + 8 + np.abs(l)) * U * np.abs(q * (l - on_lp))).sum(
        -1, keepdims=True) + np.where(rest > 0, 2 * eps * (1.0 + np.abs(gap)) + 2 * d, 0.0)
    rel = 2 * d + 6 * U * span + 24 * U
    share_rel = 2 * d + 6 * U * (np.where(share > 0, np.abs(lp - l_off), 0.0) + np.log(cols)) + 24 * U
    grad = whole * p - rest * share
    tol = p * (whole * rel + eps) + share * (rest * share_rel + eps)
    np.put_along_axis(grad, ids, whole * np.exp(on_lp) - q, -1)
    np.put_along_axis(tol, ids, np.exp(on_lp) * (whole * np.take_along_axis(rel, ids, -1) + eps) + q * U * (np.abs(l) + k + 8), -1)
    w = w.astype(np.float64)
    return (w * loss[:, 0], w[:, None] / T * grad, np.abs(w) * (loss_tol[:, 0] + U * np.abs(loss[:, 0])),
            np.abs(w)[:, None] / T * tol)


def check(pp, y, dtype, ids, lq, T, w=None):
    x = torch.from_numpy(np.ascontiguousarray(y, dtype=np.float32)).to(TYPES[dtype]).cuda()
    xd = x.double().cpu().numpy()
    w = np.ones(len(y), np.float32) if w is None else w
    loss, grad, loss_tol, grad_tol = want(xd, ids, lq, w, T)
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    got = pp.distill(x, cu(ids), cu(lq), cu(w), temperature=T, tail=True)
    a, b = got.loss.double().cpu().numpy(), got.grad.double().cpu().numpy()
    assert np.isfinite(loss).all() and np.isfinite(grad).all()
    assert np.isfinite(a).all(), f"loss {a}, {loss} expected"
    assert np.isfinite(b).all(), "gradient is not finite"
    assert (np.abs(a - loss) <= loss_tol).all(), (a, loss, loss_tol)
    # the exponentials that are flushed below 2^-126 meet coefficients of |w| / T
    tiny = max(ref.TINY[dtype], 2.0 ** -120 * np.abs(w).max() / T)
    over = np.abs(b - grad) - (grad_tol + ref.ROUND[dtype] * 1.01 * np.abs(grad) + tiny)
    assert (over <= 0).all(), f"{over.max()} above its bound"
    return got


def teacher(rows, cols, k, mass, g):
    """Distinct columns, and log probabilities that hold `mass` of each row."""
    ids = np.stack([g.permutation(cols)[:k] for _ in range(rows)])
    q = g.uniform(0.5, 1.5, (rows, k))
    return ids, np.log(q / q.sum(-1, keepdims=True) * mass).astype(np.float32)


# rows that a warp takes, that one block and that a cluster hold, and (float32, past 1 MB) that are read in tiles
COLS = [40, 1000, 7001, 40003, 300001]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cols", COLS)
def test_the_student_holds_the_teachers_columns_alone(pp, cols, dtype):
    """Everything off the teacher's columns lies `nats` below them."""
    g = np.random.default_rng(cols)
    for T, nats in ((1.0, 60.0), (1.0, 86.5), (1.0, 100.0), (1.0, 4000.0), (0.5, 120.0), (0.1, 90.0), (0.05, 200.0), (7.0, 95.0)):
        ids, lq = teacher(3, cols, 5, 0.9, g)
        y = g.normal(0.0, T, (3, cols)) - nats * T
        np.put_along_axis(y, ids, g.normal(0.0, T, ids.shape), -1)
        check(pp, y, dtype, ids, lq, T, np.array([1.0, -0.5, 3.0], np.float32))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cols", COLS)
def test_one_column_left_beside_the_teachers(pp, cols, dtype):
    """The rest of the row is masked: its gradient is 0, and all of the tail's falls on the column that is left."""
    g = np.random.default_rng(cols + 1)
    for T, nats in ((1.0, 86.0), (1.0, 87.5), (1.0, 150.0), (0.25, 89.0), (1.0, 3.0)):
        ids, lq = teacher(2, cols, 32, 0.9, g)
        y = np.full((2, cols), -np.inf)
        free = np.array([np.setdiff1d(np.arange(cols), i)[-1] for i in ids])
        y[np.arange(2), free] = -nats * T
        np.put_along_axis(y, ids, 0.0, -1)
        got = check(pp, y, dtype, ids, lq, T)
        grad = got.grad.double().cpu().numpy()
        assert np.array_equal(grad[y == -np.inf], np.zeros((y == -np.inf).sum()))
        # the gradient of a row adds up to 0
        assert np.allclose(grad.sum(-1), 0.0, atol=40 * ref.ROUND[dtype] * 0.1 / T + 1e-5 / T)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cols", COLS)
def test_the_student_holds_nothing_of_the_teachers_columns(pp, cols, dtype):
    """The other way round: the teacher's columns lie far below the others."""
    g = np.random.default_rng(cols + 2)
    for T, nats, mass in ((1.0, 100.0, 0.9), (0.1, 300.0, 0.5), (1.0, 88.0, 1e-4), (2.0, 40.0, 1.0 - 2.0 ** -18)):
        ids, lq = teacher(3, cols, 7, mass, g)
        y = g.normal(0.0, T, (3, cols))
        np.put_along_axis(y, ids, g.normal(0.0, T, ids.shape) - nats * T, -1)
        check(pp, y, dtype, ids, lq, T)


@pytest.mark.parametrize("temperature", [2.0 ** -20, 1e-3, 0.05, 17.0, 2.0 ** 20])
@pytest.mark.parametrize("cols", COLS)
def test_temperatures(pp, cols, temperature):
    """The accepted range, with logits of a fixed size and with ones that go by the temperature."""
    g = np.random.default_rng(cols + 3)
    for scale in (2.0, 5.0 * temperature):
        ids, lq = teacher(3, cols, 9, 0.8, g)
        check(pp, g.normal(0.0, scale, (3, cols)), "f32", ids, lq, temperature)


def test_the_loss_grows_with_the_gap(pp):
    """The example of one likely column: the loss is the teacher's remaining mass times the gap, and the gradient of the
    two columns off it -rest / 2 / T each."""
    ids, lq = np.array([[0]]), np.log(np.array([[0.9]], np.float32))
    for gap in (10.0, 60.0, 1000.0):
        got = check(pp, np.array([[gap, 0.0, 0.0]]), "f32", ids, lq, 0.5)
        # ln p_off = ln 2 - gap / T
        assert abs(got.loss.item() - (0.9 * np.log(0.9) + 0.1 * (np.log(0.05) + gap / 0.5))) < 1e-4 * (1 + gap)
        assert torch.allclose(got.grad[0, 1:], torch.full((2,), -0.1 / 0.5 / 2, device="cuda"), rtol=1e-5)
