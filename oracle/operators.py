"""Float64 oracle of the operators beside the layer, written from their formulas.

Layer norm (forward, and backward for given statistics), products grouped by expert (forward
and both gradients), and the orthogonalised update (Newton-Schulz products).  NumPy only; shares
no code with the GPU path.
"""
import numpy as np


def layer_norm(x, weight, bias, eps):
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    xh = (x - mean) * rstd
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def group_rows(offsets, M):
    """[(first, last)] per group: offsets clamped into [0, M] and made non-decreasing."""
    o = np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, M))
    return list(zip(o[:-1], o[1:]))


def grouped_matmul(x, w, offsets):
    """y, and which rows belong to a group (the others' y is zero)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    y = np.zeros((x.shape[0], w.shape[1]))
    inside = np.zeros(x.shape[0], bool)
    for e, (a, b) in enumerate(group_rows(offsets, x.shape[0])):
        y[a:b] = x[a:b] @ w[e].T
        inside[a:b] = True
    return y, inside


def grouped_matmul_backward(x, w, offsets, dy):
    x, w, dy = (np.asarray(t, np.float64) for t in (x, w, dy))
    dx, dw = np.zeros_like(x), np.zeros_like(w)
    for e, (a, b) in enumerate(group_rows(offsets, x.shape[0])):
        dx[a:b] = dy[a:b] @ w[e]
        dw[e] = dy[a:b].T @ x[a:b]
    return dx, dw


def orthogonalize(g, steps=5, eps=1e-7, coefficients=(3.4445, -4.7750, 2.0315), dtype=np.float64):
    """One matrix; `dtype` other than float64 evaluates the same formula in that precision."""
    a, b, c = (dtype(v) for v in coefficients)
    x = np.asarray(g, np.float64)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    norm = np.sqrt((x ** 2).sum()) + eps
    x = (x / norm if norm > 0 else x).astype(dtype)
    for _ in range(steps):
        gram = x @ x.T
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.T if tall else x
