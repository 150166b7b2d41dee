"""The float64 oracle of the dense row operators, pinned by finite differences, closed forms and planted mistakes."""
import numpy as np
import pytest

from oracle import dense


def _difference(f, a, h=1e-6):
    """Central differences of the scalar f with respect to every entry of a."""
    grad = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + h
        up = f()
        a[i] = keep - h
        down = f()
        a[i] = keep
        grad[i] = (up - down) / (2 * h)
    return grad


@pytest.mark.parametrize("activation", ["none", "silu"])
def test_linear_vjp_matches_differences(activation):
    rng = np.random.default_rng(0)
    x, W, b, r = (rng.standard_normal(s) for s in ((4, 3, 5), (5, 6), (6,), (4, 3, 6)))
    g = rng.standard_normal((4, 3, 6))
    _, z = dense.linear_forward(x, W, b, activation, r)
    grads = dense.linear_backward(x, W, g, z, activation)

    def loss():
        return float((dense.linear_forward(x, W, b, activation, r)[0] * g).sum())

    for a, got in zip((x, W, b), grads):
        want = _difference(loss, a)
        assert np.max(np.abs(got - want)) <= 1e-7 * max(1, np.max(np.abs(want)))
    # the residual's gradient is the cotangent itself
    assert np.max(np.abs(_difference(loss, r) - g)) <= 1e-7 * np.max(np.abs(g))
    # a planted mistake: the activation's derivative left out
    if activation == "silu":
        assert np.max(np.abs(dense.linear_backward(x, W, g, z, "none")[1] - grads[1])) > 1e-2


def test_layer_norm_vjp_matches_differences():
    rng = np.random.default_rng(1)
    x, w, b, g = (rng.standard_normal(s) for s in ((3, 2, 7), (7,), (7,), (3, 2, 7)))
    _, mean, rstd = dense.layer_norm_forward(x, w, b, 0.01)
    grads = dense.layer_norm_backward(x, w, mean, rstd, g)

    def loss():
        return float((dense.layer_norm_forward(x, w, b, 0.01)[0] * g).sum())

    for a, got in zip((x, w, b), grads):
        want = _difference(loss, a)
        assert np.max(np.abs(got - want)) <= 1e-7 * max(1, np.max(np.abs(want)))


def test_closed_forms():
    assert dense.act(np.array([0.0]), "silu")[0] == 0 and dense.act_grad(np.array([0.0]), "silu")[0] == 0.5
    z = np.array([-800.0, 800.0])
    assert np.array_equal(dense.act(z, "silu"), [0.0, 800.0]) and np.array_equal(dense.act_grad(z, "silu"), [0.0, 1.0])
    x = np.random.default_rng(2).standard_normal((5, 9))
    out, mean, rstd = dense.layer_norm_forward(x, eps=0.0)
    assert np.max(np.abs(out.mean(-1))) < 1e-14 and np.max(np.abs((out**2).mean(-1) - 1)) < 1e-13
    # invariant to a shift and a scale of the row, so the gradient is orthogonal to both
    gx, _, _ = dense.layer_norm_backward(x, None, mean, rstd, np.cos(x))
    assert np.max(np.abs(gx.sum(-1))) < 1e-12 and np.max(np.abs((gx * x).sum(-1))) < 1e-12
    # one channel: nothing but the bias is left
    assert np.array_equal(dense.layer_norm_forward(x[:, :1], np.array([3.0]), np.array([2.0]))[0], np.full((5, 1), 2.0))
