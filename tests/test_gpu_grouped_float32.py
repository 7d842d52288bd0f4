"""float32 grouped products over everything float32 holds: infinities, NaN and the ends of the
range, and operands whose experts, rows and channels differ by any factor.

Each test runs on both sides of the rules that send a product with few rows per group to a
path of its own (`_few`, `_few_dx`, checked against the workspace that the library asks for).

Tolerances per element, u = 2^-24, for a sum of n products: operands in three parts are exact
(a float32 value is hi + mid + lo); of the nine products of parts six are taken, the others are at
most 2^-22.99 < 2.02 u of the product; every addition rounds by at most 2 u of the partial sum,
and there are 6 (n + 8) of them: (12 (n + 8) + 3) u sum|products|, and u |result| for the store.
Operands in two float16 parts lose 2 u each and lo lo' <= 4 u of a product, 8 u where 3 u stand
above, and with half as many additions the same bound holds; what lies far below its row's
largest value is held to 2^-38 of that.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import operators as ref
from parity_helpers import say
from test_gpu_operators import U, _bits, _offsets, dev, host, mx

pytestmark = pytest.mark.gpu


def _few(M, E, n, k):
    return k % 4 == 0 and n >= 32 and M <= 64 * E


def _few_dx(M, E, n, k):
    return k % 4 == 0 and n % 4 == 0 and n >= 32 and k >= 192 and M <= E * (128 if k >= 256 else 64)


def _size(query, *args):
    out = ctypes.c_size_t(0)
    assert query(*args, ctypes.byref(out)) == 0
    return out.value


def _side(M, E, n, k, few, few_dx):
    """The shape falls on the expected side of both rules: without a prepared w the workspace
    does not grow with the experts."""
    L = mx.load_library()
    assert (_few(M, E, n, k), _few_dx(M, E, n, k)) == (few, few_dx)
    more = min(1024, 2 * E)
    assert few == (_size(L.moe_grouped_matmul_workspace_size, M, E, n, k, 0) ==
                   _size(L.moe_grouped_matmul_workspace_size, M, more, n, k, 0))
    q = L.moe_grouped_matmul_backward_workspace_size
    assert few_dx == (_size(q, M, E, n, k, 0, 1, 0) == _size(q, M, more, n, k, 0, 1, 0))


def _tol(a, b, n):
    """Tolerance of a @ b^T (absolute values) over n terms."""
    return (12 * (n + 8) + 8) * U * (a @ b.T)


def _same(got, want, tol, label):
    """NaN and infinities where the definition has them, within tol elsewhere."""
    g = host(got)
    assert (np.isnan(g) == np.isnan(want)).all(), f"{label}: NaN"
    big = np.abs(want) > 3.4028236e38                  # rounds to an infinity
    assert (np.isinf(g) == big).all() and (g[big] * want[big] > 0).all(), f"{label}: infinities"
    ok = np.isfinite(want) & ~big
    err = np.abs(np.where(ok, g, 0.0) - np.where(ok, want, 0.0))
    bad = ~(err <= np.where(ok, tol + U * np.abs(want), 1.0))
    assert not bad.any(), (label, int(bad.sum()), float(err[bad].max()))


def _check_all(x, w, off, dy, label, floor=0.0):
    """y, dx and dw against the definition in float64.  floor: of a row's largest value, for y on
    the path with two parts."""
    say(label)
    y = mx.grouped_matmul(x, w, off)
    dx, dw = mx.grouped_matmul_backward(x, w, off, dy)
    torch.cuda.synchronize()
    X, W, DY = host(x), host(w), host(dy)
    fx, fw, fdy = (np.where(np.isfinite(t), np.abs(t), 0.0) for t in (X, W, DY))
    M, k = X.shape
    n = W.shape[1]
    with np.errstate(invalid="ignore", over="ignore"):
        for e, (a, b) in enumerate(ref.group_rows(off.cpu().numpy(), M)):
            t = _tol(fx[a:b], fw[e], k)
            if floor:
                t = t + floor * (fx[a:b].max(1, initial=0)[:, None] * fw[e].sum(1) +
                                 fx[a:b].sum(1)[:, None] * fw[e].max(1))
            _same(y[a:b], X[a:b] @ W[e].T, t, f"{label} y {e}")
            _same(dx[a:b], DY[a:b] @ W[e], _tol(fdy[a:b], fw[e].T, n), f"{label} dx {e}")
            _same(dw[e], DY[a:b].T @ X[a:b], _tol(fdy[a:b].T, fx[a:b].T, b - a), f"{label} dw {e}")


# rows of the groups, n, k, and the sides of the rules: few rows, few rows with a width for y only, and for
# dx only, an odd width, many rows (tiles of 64), and of tiles of 128 and 256
SHAPES = {
    "few": ([30, 64, 0, 9], 48, 200, True, True),
    "few y": ([30, 64, 0, 9], 48, 72, True, False),
    "few dx": ([100, 200, 0, 130], 72, 260, False, True),
    "odd width": ([30, 64, 0, 9], 50, 203, False, False),
    "many rows": ([300, 150, 0, 9], 72, 200, False, False),
    "tiles of 128": ([900, 830, 0, 1100, 900], 1000, 780, False, False),
    "tiles of 256": ([1700, 1530, 0, 1100, 900], 2060, 2060, False, False),
}


def _normal(name, seed):
    sizes, n, k, few, few_dx = SHAPES[name]
    M, E = sum(sizes) + 3, len(sizes)
    _side(M, E, n, k, few, few_dx)
    r = np.random.default_rng(seed)
    x, w, dy = r.normal(size=(M, k)), 0.3 * r.normal(size=(E, n, k)), r.normal(size=(M, n))
    return x, w, torch.from_numpy(_offsets(sizes, 2)).cuda(), dy, r


@pytest.mark.parametrize("name", SHAPES)
def test_infinities_and_nan_come_out_as_in_float32(name):
    x, w, off, dy, _ = _normal(name, 1)
    last = len(w) - 1
    a = int(off[last])                                  # a row of the last group
    x[2 + 5, 7] = np.inf
    x[2 + 6, 7], x[2 + 6, 9] = np.inf, -np.inf
    x[2 + 31, 0] = np.nan
    x[a, 3] = -np.inf
    w[1, 3, 11] = -np.inf
    w[1, 4, 11] = 0.0
    w[last, -1, -1] = np.nan
    dy[2 + 12, 6] = np.inf
    dy[a + 2, 1] = -np.inf
    dy[a + 3, 1] = np.inf
    dy[a + 4] = np.nan
    _check_all(dev(x), dev(w), off, dev(dy), name, floor=2.0 ** -37)


@pytest.mark.parametrize("name", SHAPES)
def test_sums_that_leave_the_range_on_the_way(name):
    """Products past float32's range that cancel, results past it, and the largest values."""
    x, w, off, dy, _ = _normal(name, 2)
    x[2, :4], w[0, 5, :4] = [2e38, 2e38, -2e38, -2e38], [1.5, 1.5, 1.5, 1.2]
    x[3, 0], w[0, 6, 0] = 3.4e38, -3.0
    w[1, 1, 2] = 3.4028234e38                           # rounds up as a bfloat16
    x[40, 2] = 0.25
    dy[2, :4], w[0, :4, 9] = [2e38, 2e38, -2e38, -2e38], [1.5, 1.5, 1.5, 1.2]
    dy[4:8, 8], x[4:8, 1] = [2e38, 2e38, -2e38, -2e38], [1.5, 1.5, 1.5, 1.2]
    _check_all(dev(x), dev(w), off, dev(dy), name, floor=2.0 ** -37)


# ---------------------------------------------------------------- operands of uneven scale
def _check_dw(x, w, off, dy, label):
    say(label)
    _, dw = mx.grouped_matmul_backward(x, w, off, dy, need_dx=False)
    both = mx.grouped_matmul_backward(x, w, off, dy)[1]
    torch.cuda.synchronize()
    assert torch.equal(_bits(dw), _bits(both))
    X, DY = host(x), host(dy)
    for e, (a, b) in enumerate(ref.group_rows(off.cpu().numpy(), len(X))):
        t = _tol(np.abs(DY[a:b]).T, np.abs(X[a:b]).T, b - a)
        _same(dw[e], DY[a:b].T @ X[a:b], t, f"{label} dw {e}")


@pytest.mark.parametrize("name", SHAPES)
def test_weight_gradients_of_experts_rows_and_channels_of_any_scale(name):
    x, w, off, dy, r = _normal(name, 3)
    at = off.cpu().numpy()
    rows, n, k = len(x), dy.shape[1], x.shape[1]
    w = dev(w)
    # experts whose gradients differ by 2^-14 .. 2^-60, and one far above the others
    scaled = dy.copy()
    for e, p in zip(range(len(at) - 1), (0, -30, 0, -60, 20) if len(at) > 5 else (0, -30, 0, -14)):
        scaled[at[e]:at[e + 1]] *= 2.0 ** p
    _check_dw(dev(x), w, off, dev(scaled), f"{name}: experts")
    # channels of dy and of x
    sy, sx = 2.0 ** np.floor(r.uniform(-40, 20, n)), 2.0 ** np.floor(r.uniform(-40, 20, k))
    _check_dw(dev(x * sx), w, off, dev(dy * sy), f"{name}: channels")
    # rows whose dy and x are each other's opposite, and one row above all others
    s = 2.0 ** np.floor(r.uniform(-60, 60, (rows, 1)))
    _check_dw(dev(x / s), w, off, dev(dy * s), f"{name}: balanced rows")
    loud = dy.copy()
    loud[at[0] + 3] *= 2.0 ** 40
    _check_dw(dev(x), w, off, dev(loud), f"{name}: one row")
    # the smallest values: subnormal ones on one side
    _check_dw(dev(x * 2.0 ** 100), w, off, dev(dy * 2.0 ** -140), f"{name}: small dy")
    _check_dw(dev(x * 2.0 ** -140), w, off, dev(dy * 2.0 ** 100), f"{name}: small x")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", SHAPES)
def test_weight_gradients_show_bad_rows_under_a_zero_gradient(name, dtype):
    """0 x NaN and 0 x infinity are NaN: a row of x that broke shows even where dy is zero."""
    x, w, off, dy, _ = _normal(name, 4)
    x[2 + 3, 5], x[2 + 4, 6] = np.nan, np.inf
    dy[2 + 3:2 + 5] = 0.0
    x, w, dy = dev(x, dtype), dev(w, dtype), dev(dy, dtype)
    say(f"{name} {dtype}: zero gradient")
    dw = mx.grouped_matmul_backward(x, w, off, dy, need_dx=False)[1]
    torch.cuda.synchronize()
    want = torch.zeros_like(dw, dtype=torch.bool)
    want[0, :, 5:7] = True
    assert (torch.isnan(dw) == want).all() and torch.isfinite(dw[~want]).all()


@pytest.mark.parametrize("name", ["few", "few y"])
def test_few_rows_with_operands_of_any_scale(name):
    x, w, off, dy, r = _normal(name, 6)
    n, k = w.shape[1:]
    few_dx = SHAPES[name][4]

    def check(x, w, dy, label):
        say(f"{name}: {label}")
        x, w, dy = dev(x), dev(w), dev(dy)
        y = mx.grouped_matmul(x, w, off)
        dx = mx.grouped_matmul_backward(x, w, off, dy, need_dw=False)[0]
        torch.cuda.synchronize()
        X, W, DY = host(x), host(w), host(dy)
        for e, (a, b) in enumerate(ref.group_rows(off.cpu().numpy(), len(X))):
            _same(y[a:b], X[a:b] @ W[e].T, _tol(np.abs(X[a:b]), np.abs(W[e]), k), f"{label} y {e}")
            if few_dx:
                t = _tol(np.abs(DY[a:b]), np.abs(W[e]).T, n)
                _same(dx[a:b], DY[a:b] @ W[e], t, f"{label} dx {e}")

    # small weights against large rows: ordinary results out of parts near the range's end
    for p in (110, 120, 126, 138):                       # (subnormal weights from 2^-126 down)
        check(x * 2.0 ** 100, w * 2.0 ** -p, dy * 2.0 ** 100, f"weights at 2^-{p}")
    # rows, and channels of the contraction whose factors are each other's opposite
    sr = 2.0 ** np.floor(r.uniform(-60, 60, (len(x), 1)))
    check(x * sr, w, dy * sr, "rows")
    s = 2.0 ** np.floor(r.uniform(-60, 60, k))
    check(x * s, w / s, dy, "channels")
    s = 2.0 ** np.floor(r.uniform(-60, 60, n))
    check(x, w / s[:, None], dy * s, "output channels")


def _check_dx(x, w, off, dy, label):
    say(label)
    dx, _ = mx.grouped_matmul_backward(x, w, off, dy, need_dw=False)
    both = mx.grouped_matmul_backward(x, w, off, dy)[0]
    torch.cuda.synchronize()
    assert torch.equal(_bits(dx), _bits(both))
    W, DY = host(w), host(dy)
    for e, (a, b) in enumerate(ref.group_rows(off.cpu().numpy(), len(DY))):
        t = _tol(np.abs(DY[a:b]), np.abs(W[e]).T, dy.shape[1])
        _same(dx[a:b], DY[a:b] @ W[e], t, f"{label} dx {e}")


@pytest.mark.parametrize("name", SHAPES)
def test_input_gradients_through_weights_of_any_scale(name):
    x, w, off, dy, r = _normal(name, 5)
    n, k = w.shape[1:]
    x = dev(x)
    # experts, columns of w, and rows of dy
    se, sk = 2.0 ** np.array([0, -30, 20, 40, -60][:len(w)]), 2.0 ** np.floor(r.uniform(-40, 20, k))
    sr = 2.0 ** np.floor(r.uniform(-40, 20, (len(dy), 1)))
    _check_dx(x, dev(w * se[:, None, None] * sk), off, dev(dy * sr), f"{name}: experts, columns, rows")
    # output channels whose w and dy are each other's opposite, and one row of w above all others
    s = 2.0 ** np.floor(r.uniform(-60, 60, n))
    _check_dx(x, dev(w / s[:, None]), off, dev(dy * s), f"{name}: balanced channels")
    loud = w.copy()
    loud[:, 3] *= 2.0 ** 40
    _check_dx(x, dev(loud), off, dev(dy), f"{name}: one channel")


# ---------------------------------------------------------------- the path with two parts
@pytest.mark.parametrize("name", [s for s in SHAPES if not SHAPES[s][3]])
def test_products_of_rows_of_any_scale(name):
    """Rows of x and of w scaled by factors from 1e-30 to 1e20: each y keeps its own accuracy."""
    x, w, off, _, r = _normal(name, 7)
    x *= 10.0 ** r.uniform(-30, 8, (len(x), 1))
    w *= 10.0 ** r.uniform(-8, 20, (*w.shape[:2], 1))
    x, w = dev(x), dev(w)
    say(f"{name}: rows of any scale")
    y = mx.grouped_matmul(x, w, off)
    torch.cuda.synchronize()
    X, W = host(x), host(w)
    for e, (a, b) in enumerate(ref.group_rows(off.cpu().numpy(), len(X))):
        ax, aw = np.abs(X[a:b]), np.abs(W[e])
        t = _tol(ax, aw, x.shape[1]) + 2.0 ** -37.9 * (ax.max(1, initial=0)[:, None] * aw.sum(1) +
                                                       ax.sum(1)[:, None] * aw.max(1))
        _same(y[a:b], X[a:b] @ W[e].T, t, f"{name} y {e}")


def test_products_with_prepared_weights_past_4_gib():
    E, n, k = 600, 1024, 2046                            # (a width that goes without the few rows' path)
    torch.manual_seed(2)
    sizes = np.zeros(E, int)
    sizes[[0, 300, 598, 599]] = 3, 70, 1, 6
    M = int(sizes.sum())
    _side(M, E, n, k, False, False)
    x, w = torch.randn(M, k, device="cuda"), torch.randn(E, n, k, device="cuda")
    dy = torch.randn(M, n, device="cuda")
    off = torch.from_numpy(_offsets(sizes)).cuda()
    say("grouped f32, w of 5 GB and its parts")
    y = mx.grouped_matmul(x, w, off)
    dx, dw = mx.grouped_matmul_backward(x, w, off, dy)
    torch.cuda.synchronize()
    for e, (a, b) in enumerate(ref.group_rows(off.cpu().numpy(), M)):
        if a < b:
            X, W, DY = host(x[a:b]), host(w[e]), host(dy[a:b])
            ax, aw, ady = np.abs(X), np.abs(W), np.abs(DY)
            _same(y[a:b], X @ W.T, _tol(ax, aw, k), f"y {e}")
            _same(dx[a:b], DY @ W, _tol(ady, aw.T, n), f"dx {e}")
            _same(dw[e], DY.T @ X, _tol(ady.T, ax.T, b - a), f"dw {e}")
    assert not dw[1:300].any() and not dw[301:598].any()


# ---------------------------------------------------------------- on both sides of the rules
@pytest.mark.parametrize("name", SHAPES)
def test_bad_offsets_are_clamped(name):
    x, w, _, dy, _ = _normal(name, 8)
    x, w, dy, M = dev(x), dev(w), dev(dy), len(x)
    a, b = M // 3, M // 2
    bad, good = [-9, a, a - 5, M + 1000], [0, a, a, M]
    tail = len(w) + 1 - len(bad)
    say(f"{name}: bad offsets")
    res = []
    for o in (bad + [b] * tail, good + [M] * tail):
        o = torch.tensor(o, dtype=torch.int32, device="cuda")
        res.append((mx.grouped_matmul(x, w, o), *mx.grouped_matmul_backward(x, w, o, dy)))
    torch.cuda.synchronize()
    for p, q in zip(*res):
        assert torch.equal(_bits(p), _bits(q))


def _all_calls(ws=None):
    calls = []
    for name in SHAPES:
        if not name.startswith("tiles"):
            x, w, off, dy, _ = _normal(name, 9)
            x, w, dy = dev(x), dev(w), dev(dy)
            calls += [lambda x=x, w=w, off=off: (mx.grouped_matmul(x, w, off, workspace=ws),),
                      lambda x=x, w=w, off=off, dy=dy: mx.grouped_matmul_backward(x, w, off, dy, workspace=ws),
                      lambda x=x, w=w, off=off, dy=dy: mx.grouped_matmul_backward(
                          x, w, off, dy, need_dw=False, workspace=ws)[:1]]
    return calls


@pytest.mark.parametrize("shared", [False, True])
def test_repeated_on_another_stream_and_captured(shared):
    """Every path's calls, with a workspace each or one that all graphs share: the same bits on
    another stream and in graphs replayed in changing order with eager calls between."""
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda") if shared else None
    calls = _all_calls(ws)
    want = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [c() for c in calls]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for g, v in zip(got, want):
        assert all(torch.equal(_bits(p), _bits(q)) for p, q in zip(g, v))
    graphs, outs = [], []
    for i, c in enumerate(calls):
        say(f"capture {i}")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    order = np.random.default_rng(10)
    for k in range(3):
        if shared:
            ws.fill_(255)                        # what other calls left there does not matter
        for i in order.permutation(len(calls)):
            for t in outs[i]:
                t.zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(_bits(p), _bits(q)) for p, q in zip(outs[i], want[i])), (k, i)
            assert all(torch.equal(_bits(p), _bits(q)) for p, q in zip(calls[i](), want[i])), (k, i)
