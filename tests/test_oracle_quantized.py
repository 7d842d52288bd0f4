"""Pins of the float64 oracle behind the 8-bit experts and the balance loss (CPU): closed forms,
every 8-bit value against PyTorch's own conversion, central differences for every gradient."""
import numpy as np
import pytest
import torch

from oracle import operators as ops

RNG = np.random.default_rng
KINDS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, dn = x.copy(), x.copy()
        up[i] += h
        dn[i] -= h
        g[i] = (f(up) - f(dn)) / (2 * h)
    return g


def test_rms_norm_closed_form():
    y, rstd = ops.rms_norm([[3.0, 4.0], [0.0, 0.0]], [2.0, 1.0], 0.5)
    assert np.allclose(rstd, [1 / np.sqrt(13.0), np.sqrt(2.0)])
    assert np.allclose(y, [[6 / np.sqrt(13), 4 / np.sqrt(13)], [0, 0]])


@pytest.mark.parametrize("weight", [True, False])
def test_rms_norm_gradients_are_the_differences(weight):
    r = RNG(1)
    h, dy, dh = r.normal(size=(4, 7)), r.normal(size=(4, 7)), r.normal(size=(4, 7))
    w = r.normal(size=7) if weight else None
    dx, dw = ops.rms_norm_backward(dy, h, w, ops.rms_norm(h, w, 1e-3)[1], dh)

    def loss(h_, w_):
        return (dy * ops.rms_norm(h_, w_, 1e-3)[0]).sum() + (dh * h_).sum()

    assert np.allclose(dx, _differences(lambda v: loss(v, w), h), atol=1e-6)
    assert np.allclose(dw, _differences(lambda v: loss(h, v), np.ones(7) if w is None else w), atol=1e-6)


@pytest.mark.parametrize("kind", KINDS)
def test_rounding_to_eight_bits(kind):
    t = KINDS[kind]
    every = torch.arange(256, dtype=torch.uint8).view(t).double()
    every = every[torch.isfinite(every)].sort().values.numpy()
    assert np.abs(every).max() == ops.F8[kind][2]
    assert (ops.round_f8(every, kind) == every).all()                # each stands for itself
    mid = (every[1:] + every[:-1]) / 2                               # ties, and beside them
    for v in (mid, mid * (1 + 1e-7), mid * (1 - 1e-7), RNG(2).normal(size=4000) * 50):
        want = torch.from_numpy(v.astype(np.float32)).to(t).double().numpy()
        assert (ops.round_f8(v.astype(np.float32), kind) == want).all()


def test_scales_of_blocks():
    x = np.zeros((2, 300))
    x[0, 5], x[0, 130], x[0, 299] = -448.0, 7.0, np.inf
    x[1, 128:256] = 1e-44
    s = ops.block_scales(x, "e4m3")
    assert s.shape == (2, 3)
    assert s[0].tolist() == [1.0, 7 / 448, 1.0] and s[1].tolist() == [1.0, 2.0 ** -126, 1.0]
    w = np.zeros((2, 130, 257))
    w[1, 129, 256] = 2.0
    m = ops.matrix_scales(w, "e5m2")
    assert m.shape == (2, 2, 3) and m[1, 1, 2] == 2 / 57344 and (m.reshape(-1)[:-1] == 1).all()


def test_quantized_products_are_products_of_what_the_values_stand_for():
    r = RNG(3)
    x, w, xs, ws = r.normal(size=(5, 130)), r.normal(size=(2, 3, 130)), r.random((5, 2)), r.random((2, 1, 2))
    y, _ = ops.grouped_matmul_quantized(x, xs, w, ws, [0, 2, 5])
    by_hand = sum(x[4, j] * xs[4, j // 128] * w[1, 2, j] * ws[1, 0, j // 128] for j in range(130))
    assert np.isclose(y[4, 2], by_hand)
    dy, dys = r.normal(size=(5, 3)), r.random((5, 1))
    dx, _ = ops.grouped_matmul_quantized_dx(dy, dys, w, ws, [0, 2, 5])
    by_hand = sum(dy[1, i] * dys[1, 0] * w[0, i, 129] * ws[0, 0, 1] for i in range(3))
    assert np.isclose(dx[1, 129], by_hand)


def _softmax(z):
    e = np.exp(z - z.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def test_balance_loss_of_the_batch_is_the_balance_statistics():
    import oracle
    r = RNG(4)
    scores = _softmax(r.normal(size=(40, 8)))
    idx = np.argsort(-scores, 1)[:, :3]
    groups = [0, 0, 1, 1, 1, 2, 2, 2]
    got = ops.balance_loss(scores, idx, None, None, groups, 3, 0.7, 0.4)
    want = oracle.balance_statistics(scores, idx, 3, [[0, 1], [2, 3, 4], [5, 6, 7]], 0.7, 0.4)
    assert np.allclose(got["losses"][0], [want["L_ExpBal"], want["L_DevBal"]])
    assert np.allclose(got["P"][0], want["P"])


def test_balance_loss_closed_forms():
    # every token on expert 0 of 4 with score 1: f = (4, 0, 0, 0), P = (1, 0, 0, 0)
    scores, idx = np.tile([1.0, 0, 0, 0], (6, 1)), np.zeros((6, 1), int)
    out = ops.balance_loss(scores, idx, [0, 2, 2, 6], None, [0, 0, 1, 1], 2, 1.0, 1.0)
    assert out["counts"].tolist() == [[2, 0, 0, 0], [0, 0, 0, 0], [4, 0, 0, 0]]
    assert np.allclose(out["losses"], [[4, 2], [0, 0], [4, 2]])
    out = ops.balance_loss(scores, idx, None, [0, 0, 0, 0, 0, 0])
    assert not out["losses"].any() and not out["slopes"].any()


def test_balance_loss_gradient_is_the_difference():
    r = RNG(5)
    z = r.normal(size=(9, 5))
    idx = np.argsort(-_softmax(z), 1)[:, :2]
    offsets, mask = [1, 4, 4, 8], np.array([1, 1, 0, 1, 1, 1, 1, 0, 1], bool)
    args = dict(device_of=[0, 1, 1, 0, 7], devices=2, alpha1=0.3, alpha2=0.9)
    dl = r.normal(size=(3, 2))

    def loss(z_):
        return (dl * ops.balance_loss(_softmax(z_), idx, offsets, mask, **args)["losses"]).sum()

    s = _softmax(z)
    slopes = ops.balance_loss(s, idx, offsets, mask, **args)["slopes"]
    got = ops.balance_loss_backward(s, slopes, dl, offsets, mask)
    assert np.allclose(got, _differences(loss, z), atol=1e-7)
    assert not got[[0, 2, 7, 8]].any()
