"""Pins of the operators' float64 oracle (CPU): central differences for every gradient, closed
forms, and the singular values that Newton-Schulz products must map by their polynomial."""
import numpy as np
import pytest

from oracle import operators as ops

RNG = np.random.default_rng


def _differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, dn = x.copy(), x.copy()
        up[i] += h
        dn[i] -= h
        g[i] = (f(up) - f(dn)) / (2 * h)
    return g


def test_layer_norm_closed_form():
    y, mean, rstd = ops.layer_norm([[1.0, 3.0], [2.0, 2.0]], [2.0, 1.0], [0.5, 0.0], 0.0 + 1e-30)
    assert np.allclose(mean, [2, 2]) and np.allclose(rstd[0], 1.0)
    assert np.allclose(y[0], [-2 + 0.5, 1.0])
    assert np.allclose(y[1], [0.5, 0.0])          # a constant row has no deviations


@pytest.mark.parametrize("weight", [True, False])
def test_layer_norm_gradients_are_the_differences(weight):
    r = RNG(3)
    x, dy = r.normal(size=(4, 7)), r.normal(size=(4, 7))
    w = r.normal(size=7) if weight else None
    b = r.normal(size=7)
    _, mean, rstd = ops.layer_norm(x, w, b, 1e-3)
    dx, dw, db = ops.layer_norm_backward(dy, x, w, mean, rstd)

    def loss(x_, w_, b_):
        return (dy * ops.layer_norm(x_, w_, b_, 1e-3)[0]).sum()

    assert np.allclose(dx, _differences(lambda v: loss(v, w, b), x), atol=1e-6)
    one = np.ones(7) if w is None else w
    assert np.allclose(dw, _differences(lambda v: loss(x, v, b), one), atol=1e-6)
    assert np.allclose(db, _differences(lambda v: loss(x, w, v), b), atol=1e-6)


def test_grouped_rows_and_gradients():
    r = RNG(4)
    x, w = r.normal(size=(9, 5)), r.normal(size=(4, 3, 5))
    offsets = [1, 3, 3, 7, 8]                    # an empty group, rows left over on both sides
    y, inside = ops.grouped_matmul(x, w, offsets)
    assert inside.tolist() == [False] + [True] * 7 + [False]
    assert np.allclose(y[1], w[0] @ x[1]) and np.allclose(y[7], w[3] @ x[7])
    assert not y[0].any() and not y[8].any()
    dy = r.normal(size=y.shape)
    dx, dw = ops.grouped_matmul_backward(x, w, offsets, dy)
    assert np.allclose(dx, _differences(lambda v: (dy * ops.grouped_matmul(v, w, offsets)[0]).sum(), x),
                       atol=1e-6)
    assert np.allclose(dw, _differences(lambda v: (dy * ops.grouped_matmul(x, v, offsets)[0]).sum(), w),
                       atol=1e-6)
    assert not dw[1].any()


def test_group_rows_of_bad_offsets():
    assert ops.group_rows([-4, 3, 2, 99, 5], 8) == [(0, 3), (3, 3), (3, 8), (8, 8)]


@pytest.mark.parametrize("shape", [(6, 9), (9, 6), (5, 5), (1, 4)])
def test_orthogonalize_maps_singular_values(shape):
    r = RNG(5)
    g = r.normal(size=shape)
    out = ops.orthogonalize(g, steps=5, eps=0.0)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / np.sqrt((s ** 2).sum())
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    assert np.allclose(out, (u * s) @ vt, atol=1e-9)
    assert (s > 0.6).all() and (s < 1.3).all()


def test_orthogonalize_zero_and_scale():
    assert not ops.orthogonalize(np.zeros((3, 4))).any()
    g = RNG(6).normal(size=(4, 6))
    assert np.allclose(ops.orthogonalize(g, eps=0.0), ops.orthogonalize(1e-12 * g, eps=0.0))
