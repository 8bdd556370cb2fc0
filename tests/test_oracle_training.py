"""The training operators' fp64 reference against central differences and closed forms."""
import numpy as np
import pytest

from oracle import training


def _difference(f, x, direction, h=1e-5):
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


@pytest.mark.parametrize("seed", range(3))
def test_embedding_gradient_is_the_transposed_lookup(seed):
    rng = np.random.default_rng(seed)
    tokens = np.array([3, 0, 3, -1, 7, 3, 4])  # one padding, one outside a table of 7 rows
    table, dout = rng.standard_normal((7, 5)), rng.standard_normal((7, 5))
    grad, size, count = training.embedding_grad(dout, tokens, 7, 2.5)
    way = rng.standard_normal((7, 5))
    d = _difference(lambda t: (training.embedding(t, tokens, 2.5) * dout).sum(), table, way)
    assert abs(d - (grad * way).sum()) < 1e-8
    assert count.tolist() == [1, 0, 0, 3, 1, 0, 0] and (size >= np.abs(grad)).all()


@pytest.mark.parametrize("seed", range(3))
def test_layer_norm_gradients_against_differences(seed):
    rng = np.random.default_rng(seed)
    x, dy = rng.standard_normal((4, 9)) + 1.5, rng.standard_normal((4, 9))
    w, b = rng.standard_normal(9), rng.standard_normal(9)
    _, mean, rstd = training.layer_norm(x, w, b)
    dx, dw, db = training.layer_norm_grad(dy, x, mean, rstd, w)
    for grad, f, at in ((dx, lambda v: training.layer_norm(v, w, b)[0], x),
                        (dw, lambda v: training.layer_norm(x, v, b)[0], w),
                        (db, lambda v: training.layer_norm(x, w, v)[0], b)):
        way = rng.standard_normal(at.shape)
        d = _difference(lambda v: (f(v) * dy).sum(), at, way)
        assert abs(d - (grad * way).sum()) < 1e-7 * (1 + abs(d))


@pytest.mark.parametrize("temperature", [0.5, 1.0, 3.0])
def test_distillation_gradient_against_differences(temperature):
    rng = np.random.default_rng(4)
    z, a = rng.standard_normal((5, 11)), rng.standard_normal((5, 3))
    ids = np.array([[1, 4, 7], [0, 0, 5], [10, -1, 11], [-1, 99, -7], [2, 3, 4]])
    w = np.array([0.3, 1.0, 0.7, 2.0, 0.0])
    grad = training.distill_grad(z, a, ids, w, temperature)
    way = rng.standard_normal(z.shape)
    d = _difference(lambda v: (training.distill(v, a, ids, temperature)[0] * w).sum(), z, way)
    assert abs(d - (grad * way).sum()) < 1e-8 * (1 + abs(d))
    assert not grad[3].any() and not grad[4].any()  # no live entry; weight 0
    np.testing.assert_allclose(grad.sum(1), 0.0, atol=1e-14)


def test_one_teacher_entry_is_cross_entropy():
    rng = np.random.default_rng(5)
    z = rng.standard_normal((3, 6))
    loss, _, _ = training.distill(z, np.zeros((3, 1)), np.array([[2], [0], [5]]))
    want = np.log(np.exp(z).sum(1)) - z[np.arange(3), [2, 0, 5]]
    np.testing.assert_allclose(loss, want, rtol=1e-14)


def test_equal_distributions_have_no_loss():
    rng = np.random.default_rng(6)
    z = rng.standard_normal((3, 6))
    loss, _, _ = training.distill(z, z, np.tile(np.arange(6), (3, 1)), 2.0)
    np.testing.assert_allclose(loss, 0.0, atol=1e-14)
