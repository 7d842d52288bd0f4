"""Float64 oracle of the operators beside the layer, written from their formulas.

Layer norm (forward, and backward for given statistics), products grouped by expert (forward
and both gradients), and the orthogonalised update (Newton-Schulz products); root-mean-square
norm, 8-bit values with a scale for each block of 128 and the grouped products of such values,
and the balance loss per sequence with its gradient.  NumPy only; shares no code with the GPU
path.
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


def rms_norm(h, weight, eps):
    """(y, rstd) of the rows of h."""
    h = np.asarray(h, np.float64)
    rstd = 1.0 / np.sqrt((h ** 2).mean(1) + eps)
    y = h * rstd[:, None]
    return (y if weight is None else y * np.asarray(weight, np.float64)), rstd


def rms_norm_backward(dy, h, weight, rstd, dh=None):
    """(dx, dweight) for a given rstd."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    hh = h * np.asarray(rstd, np.float64)[:, None]
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = np.asarray(rstd, np.float64)[:, None] * (g - hh * (g * hh).mean(1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * hh).sum(0)


# ---- 8 bits: name -> (bits of mantissa, exponent of the smallest normal number, largest value)
F8 = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}
BLOCK = 128


def round_f8(v, kind):
    """The 8-bit value nearest to v, ties to even (|v| below half a step past the largest)."""
    bits, low, most = F8[kind]
    v = np.asarray(v, np.float64)
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -200))), low)
    step = 2.0 ** (e - bits)
    out = np.round(v / step) * step                # numpy rounds halves to even
    assert not (np.abs(out) > most).any()
    return out


def _tops(x, axes):
    return np.where(np.isfinite(x), np.abs(x), 0.0).max(axes)


def _scales(top, kind):
    return np.where(top > 0, np.maximum(top / F8[kind][2], 2.0 ** -126), 1.0)


def block_scales(x, kind):
    """Scales of rows [T][d]: one for each 128 columns."""
    x = np.asarray(x, np.float64)
    cuts = range(0, x.shape[1], BLOCK)
    return _scales(np.stack([_tops(x[:, c:c + BLOCK], 1) for c in cuts], 1), kind)


def matrix_scales(w, kind):
    """Scales of matrices [E][n][k]: one for each 128 x 128."""
    w = np.asarray(w, np.float64)
    rows, cols = range(0, w.shape[1], BLOCK), range(0, w.shape[2], BLOCK)
    top = [[_tops(w[:, r:r + BLOCK, c:c + BLOCK], (1, 2)) for c in cols] for r in rows]
    return _scales(np.moveaxis(np.array(top), 2, 0), kind)


def spread_rows(scales, d):
    return np.repeat(np.asarray(scales, np.float64), BLOCK, -1)[..., :d]


def spread_matrix(scales, n, k):
    return np.repeat(spread_rows(scales, k), BLOCK, -2)[..., :n, :]


def grouped_matmul_quantized(x, xs, w, ws, offsets):
    """y and the sums of |products|, per element."""
    x = np.asarray(x, np.float64) * spread_rows(xs, x.shape[1])
    w = np.asarray(w, np.float64) * spread_matrix(ws, *w.shape[1:])
    return grouped_matmul(x, w, offsets)[0], grouped_matmul(abs(x), abs(w), offsets)[0]


def grouped_matmul_quantized_dx(dy, dys, w, ws, offsets):
    dy = np.asarray(dy, np.float64) * spread_rows(dys, dy.shape[1])
    w = np.swapaxes(np.asarray(w, np.float64) * spread_matrix(ws, *w.shape[1:]), 1, 2)
    return grouped_matmul(dy, w, offsets)[0], grouped_matmul(abs(dy), abs(w), offsets)[0]


def balance_loss(scores, idx, offsets=None, mask=None, device_of=None, devices=0, alpha1=1.0,
                 alpha2=1.0):
    """dict of counts, P, losses and slopes [S][2][N]: d losses / d scores of each row that counts."""
    scores, idx = np.asarray(scores, np.float64), np.asarray(idx)
    T, N = scores.shape
    K = idx.shape[1]
    spans = group_rows([0, T] if offsets is None else offsets, T)
    keep = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    out = dict(counts=np.zeros((len(spans), N), np.int64), P=np.zeros((len(spans), N)),
               losses=np.zeros((len(spans), 2)), slopes=np.zeros((len(spans), 2, N)))
    for s, (a, b) in enumerate(spans):
        rows = np.arange(a, b)[keep[a:b]]
        if not len(rows):
            continue
        for e in idx[rows].reshape(-1):
            if 0 <= e < N:
                out["counts"][s, e] += 1
        f = N * out["counts"][s] / (K * len(rows))
        out["P"][s] = P = scores[rows].mean(0)
        fd = np.zeros(N)
        for g in range(devices if device_of is not None else 0):
            of = np.asarray(device_of) == g
            if of.any():
                fd[of] = f[of].mean()
        out["losses"][s] = alpha1 * (f * P).sum(), alpha2 * (fd * P).sum()
        out["slopes"][s] = alpha1 * f / len(rows), alpha2 * fd / len(rows)
    return out


def balance_loss_backward(scores, slopes, dlosses=None, offsets=None, mask=None):
    scores, slopes = np.asarray(scores, np.float64), np.asarray(slopes, np.float64)
    T, N = scores.shape
    d = np.ones((len(slopes), 2)) if dlosses is None else np.asarray(dlosses, np.float64)
    z = np.zeros((T, N))
    for s, (a, b) in enumerate(group_rows([0, T] if offsets is None else offsets, T)):
        c = d[s] @ slopes[s]
        for t in range(a, b):
            if mask is None or mask[t]:
                z[t] = scores[t] * (c - scores[t] @ c)
    return z
