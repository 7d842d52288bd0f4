"""GPU parity of the operators beside the layer against their float64 oracle.

Tolerances, per element, u = 2^-24:
  sums    a sum of n products is off by at most (n + 8) 2 u sum|products| in any order, each
          addition by at most one unit (2 u) whatever way the matrix instructions round; the
          two-float16 split of a float32 adds at most 3 u per product (representation 2 u,
          the left-out lo lo' product u) and 2^-38 of the largest product for values far below
          their row's largest;
  stats   a row sum goes through at most 64 additions in a thread and 26 across threads: 96 u;
  store   half a step of the stored type, relative: 2^-8 for bfloat16, u for float32.
"""
import numpy as np
import pytest
import torch

from oracle import operators as ref
from parity_helpers import say

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mixture_experts_ffn_fp32_amd")

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
STORE = {"f32": U, "bf16": 2.0 ** -8}


def dev(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(DT[dtype])


def host(t):
    return t.double().cpu().numpy()


def within(got, want, tol, label):
    err = np.abs(host(got) - want) if torch.is_tensor(got) else np.abs(got - want)
    bad = ~(err <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err / np.maximum(tol, 1e-300), 0)), err.shape)
        raise AssertionError(f"{label}: {bad.sum()} of {bad.size} beyond tolerance, worst at {i}: "
                             f"error {err[i]:.3e}, tolerance {np.broadcast_to(tol, err.shape)[i]:.3e}")


# ---------------------------------------------------------------- layer norm
NORM_SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 64), (2, 513), (4, 512), (7, 1000), (33, 1024),
               (9, 1283), (6, 2050), (5, 4096), (3, 5001), (2, 8192), (2, 20000), (1, 70000),
               (700, 72), (2051, 130)]


def _norm_inputs(T, d, dtype, seed):
    r = np.random.default_rng(seed)
    x = dev(r.normal(size=(T, d)) * (1 + 3 * r.random((T, 1))) + 2 * r.normal(size=(T, 1)), dtype)
    w = dev(1 + 0.3 * r.normal(size=d), dtype)
    b = dev(0.5 * r.normal(size=d), dtype)
    return x, w, b, dev(r.normal(size=(T, d)), dtype)


def _norm_check(x, w, b, eps, dtype, label):
    y, mean, rstd = mx.layer_norm(x, w, b, eps)
    torch.cuda.synchronize()
    xh_, wh, bh = host(x), None if w is None else host(w), None if b is None else host(b)
    ry, rmean, rrstd = ref.layer_norm(xh_, wh, bh, eps)
    S = 96 * U
    emean = S * np.abs(xh_).mean(1)
    within(mean, rmean, emean + 1e-300, label + " mean")
    # var + eps = 1 / rstd^2: off by 2 |deviation| of the mean and the sum's rounding
    dev_abs = np.abs(xh_ - rmean[:, None]).mean(1)
    evar = (2 * emean + 4 * U * np.abs(xh_).max(1)) * dev_abs + emean ** 2 + 2 * S / rrstd ** 2
    erstd = rrstd * (0.5 * evar * rrstd ** 2 * 1.5 + 4 * U)
    within(rstd, rrstd, erstd, label + " rstd")
    xh = (xh_ - rmean[:, None]) * rrstd[:, None]
    exh = (emean[:, None] + 2 * U * np.abs(xh_)) * rrstd[:, None] + np.abs(xh) * (erstd / rrstd)[:, None]
    W = np.ones(x.shape[1]) if wh is None else np.abs(wh)
    B = np.zeros(x.shape[1]) if bh is None else np.abs(bh)
    tol = W * exh + 6 * U * (np.abs(xh) * W + B)
    within(y, ry, tol + STORE[dtype] * (np.abs(ry) + tol), label + " y")
    return mean, rstd


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", NORM_SHAPES)
def test_layer_norm(T, d, dtype):
    say(f"layer_norm T={T} d={d} {dtype}")
    x, w, b, dy = _norm_inputs(T, d, dtype, T * 31 + d)
    mean, rstd = _norm_check(x, w, b, 1e-5, dtype, "weights")
    _norm_check(x, None, None, 1e-2, dtype, "no weights")
    _norm_backward_check(dy, x, w, mean, rstd, dtype, "weights")
    _norm_backward_check(dy, x, None, mean, rstd, dtype, "no weights")


def _norm_backward_check(dy, x, w, mean, rstd, dtype, label):
    say(f"layer_norm_backward {tuple(x.shape)} {dtype} {label}")
    dx, dw, db = mx.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    dyh, xh_, wh = host(dy), host(x), None if w is None else host(w)
    m, rs = host(mean), host(rstd)
    rdx, rdw, rdb = ref.layer_norm_backward(dyh, xh_, wh, m, rs)
    xh = (xh_ - m[:, None]) * rs[:, None]
    exh = 3 * U * (np.abs(xh_) + np.abs(m)[:, None]) * rs[:, None]
    g = dyh if wh is None else dyh * wh
    S = 100 * U
    e1 = S * np.abs(g).mean(1)
    e2 = (S * np.abs(g * xh) + np.abs(g) * exh).mean(1)
    c1, c2 = g.mean(1), (g * xh).mean(1)
    tol = rs[:, None] * (e1[:, None] + np.abs(xh) * e2[:, None] + exh * np.abs(c2)[:, None] +
                         6 * U * (np.abs(g) + np.abs(c1)[:, None] + np.abs(xh * c2[:, None])))
    within(dx, rdx, tol + STORE[dtype] * (np.abs(rdx) + tol), label + " dx")
    n = x.shape[0] + 8
    within(dw, rdw, (n * U * np.abs(dyh * xh) + np.abs(dyh) * exh).sum(0), label + " dweight")
    within(db, rdb, n * U * np.abs(dyh).sum(0), label + " dbias")


def test_layer_norm_constant_rows_and_large_offsets():
    say("layer_norm constant rows")
    x = dev(np.full((4, 512), 3.0))
    y, mean, rstd = mx.layer_norm(x, None, None, 1e-5)
    assert torch.equal(y, torch.zeros_like(y)) and (mean == 3.0).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    r = np.random.default_rng(1)
    _norm_check(dev(1000 + r.normal(size=(5, 2048))), None, None, 1e-5, "f32", "offset 1000")


def test_layer_norm_keeps_a_bad_row_to_itself():
    r = np.random.default_rng(2)
    a = r.normal(size=(6, 256))
    clean = mx.layer_norm(dev(a))[0]
    a[2, 5] = np.nan
    a[4, 7] = np.inf
    y, mean, _ = mx.layer_norm(dev(a))
    torch.cuda.synchronize()
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).all()


# ---------------------------------------------------------------- grouped products
def _offsets(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


# sizes of the groups, rows before and behind them, n, k
GROUPED = [
    ([1], 0, 0, 1, 1),
    ([1], 0, 0, 64, 64),
    ([3], 0, 2, 8, 24),
    ([5, 0, 7], 1, 3, 17, 33),
    ([0, 0, 0], 2, 2, 16, 16),
    ([64] * 4, 0, 0, 128, 128),
    ([130, 0, 257, 1, 300], 0, 5, 200, 136),
    ([600, 1, 0, 90], 0, 0, 320, 448),
    ([1] * 40 + [0] * 20 + [3] * 9, 0, 1, 96, 192),
    ([0] * 500 + [2] + [0] * 300 + [9] + [1] * 222, 0, 0, 40, 72),
    ([7, 2, 0, 19], 0, 0, 1408, 256),
    ([6] * 12, 0, 0, 256, 704),
    ([33, 70], 0, 0, 65, 1001),
    ([1500, 700], 3, 9, 260, 520),
]


def _grouped_inputs(sizes, before, behind, n, k, dtype, seed):
    r = np.random.default_rng(seed)
    M = before + sum(sizes) + behind
    x, dy = r.normal(size=(M, k)), r.normal(size=(M, n))
    w = 0.3 * r.normal(size=(len(sizes), n, k))
    off = _offsets(sizes, before)
    outside = np.r_[0:before, before + sum(sizes):M]
    x[outside] = np.nan                     # rows outside every group are not read
    dy[outside] = np.nan
    return dev(x, dtype), dev(w, dtype), torch.from_numpy(off).cuda(), dev(dy, dtype), outside


def _sum_tol(a, b, n, dtype):
    """Tolerance of the products a @ b^T (absolute values given) over n terms."""
    t = (2 * (n + 8) * U) * (a @ b.T)
    if dtype == "f32":
        t = t + 3 * U * (a @ b.T) + n * 2.0 ** -37 * a.max(initial=0) * b.max(initial=0)
    return t


def _grouped_check(sizes, before, behind, n, k, dtype, seed=7):
    x, w, off, dy, outside = _grouped_inputs(sizes, before, behind, n, k, dtype, seed)
    say(f"grouped_matmul M={x.shape[0]} E={len(sizes)} n={n} k={k} {dtype}")
    y = mx.grouped_matmul(x, w, off)
    mark = torch.full_like(y, 7.0)
    kept = mx.grouped_matmul(x, w, off, out=mark)
    torch.cuda.synchronize()
    say("grouped_matmul_backward")
    dx, dw = mx.grouped_matmul_backward(x, w, off, dy)
    torch.cuda.synchronize()
    xh, wh, dyh = (np.nan_to_num(host(t)) for t in (x, w, dy))
    ry, inside = ref.grouped_matmul(xh, wh, off.cpu().numpy())
    rdx, rdw = ref.grouped_matmul_backward(xh, wh, off.cpu().numpy(), dyh)
    assert kept is mark
    assert not host(y)[outside].any() and not host(dx)[outside].any()
    assert (host(kept)[outside] == 7.0).all()
    ins = torch.from_numpy(inside).cuda()
    assert torch.equal(kept[ins], y[ins])
    dwf = 2.0 ** -37 * np.abs(dyh).max(initial=0) * np.abs(xh).max(initial=0)
    for e, (a, b) in enumerate(ref.group_rows(off.cpu().numpy(), x.shape[0])):
        ax, aw, ady = np.abs(xh[a:b]), np.abs(wh[e]), np.abs(dyh[a:b])
        t = _sum_tol(ax, aw, k, dtype)
        within(host(y)[a:b], ry[a:b], t + STORE[dtype] * (np.abs(ry[a:b]) + t), f"y of group {e}")
        t = _sum_tol(ady, aw.T, n, dtype)
        within(host(dx)[a:b], rdx[a:b], t + STORE[dtype] * (np.abs(rdx[a:b]) + t), f"dx of group {e}")
        t = _sum_tol(ady.T, ax.T, b - a, dtype) + (b - a) * dwf * (dtype == "f32")
        within(host(dw)[e], rdw[e], t + U * np.abs(rdw[e]), f"dw of group {e}")
        if a == b:
            assert not host(dw)[e].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped(case, dtype):
    _grouped_check(*GROUPED[case], dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grouped_bad_offsets_are_clamped(dtype):
    r = np.random.default_rng(3)
    x, w = dev(r.normal(size=(50, 64)), dtype), dev(r.normal(size=(4, 48, 64)), dtype)
    bad = np.array([-9, 20, 10, 1000, 30], np.int32)
    good = np.array([0, 20, 20, 50, 50], np.int32)
    dy = dev(r.normal(size=(50, 48)), dtype)
    say(f"grouped bad offsets {dtype}")
    res = []
    for off in (bad, good):
        o = torch.from_numpy(off).cuda()
        res.append((mx.grouped_matmul(x, w, o), *mx.grouped_matmul_backward(x, w, o, dy)))
    torch.cuda.synchronize()
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_grouped_empty_batch():
    say("grouped M = 0")
    w = torch.randn(3, 16, 24, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = torch.empty(0, 24, device="cuda"), torch.empty(0, 16, device="cuda")
    assert mx.grouped_matmul(x, w, off).shape == (0, 16)
    for dt in (torch.float32, torch.bfloat16):
        dx, dw = mx.grouped_matmul_backward(x.to(dt), w.to(dt), off, dy.to(dt))
        torch.cuda.synchronize()
        assert dx.shape == (0, 24) and not dw.any() and dw.shape == w.shape


def test_grouped_one_gradient_only():
    x, w, off, dy, _ = _grouped_inputs([9, 0, 40], 0, 0, 72, 80, "bf16", 5)
    both = mx.grouped_matmul_backward(x, w, off, dy)
    dx, none = mx.grouped_matmul_backward(x, w, off, dy, need_dw=False)
    none2, dw = mx.grouped_matmul_backward(x, w, off, dy, need_dx=False)
    torch.cuda.synchronize()
    assert none is None and none2 is None
    assert torch.equal(both[0], dx) and torch.equal(both[1], dw)


def test_grouped_f32_rows_of_any_scale():
    """Rows of x and w scaled by factors from 1e-30 to 1e30: each y keeps its own accuracy."""
    r = np.random.default_rng(11)
    M, E, n, k = 60, 3, 40, 96
    sx, sw = 10.0 ** r.uniform(-30, 8, (M, 1)), 10.0 ** r.uniform(-8, 20, (E, n, 1))
    x, w = dev(r.normal(size=(M, k)) * sx), dev(r.normal(size=(E, n, k)) * sw)
    off = torch.from_numpy(_offsets([20, 15, 25])).cuda()
    say("grouped f32 scales")
    y = mx.grouped_matmul(x, w, off)
    torch.cuda.synchronize()
    ry, _ = ref.grouped_matmul(host(x), host(w), off.cpu().numpy())
    for e, (a, b) in enumerate(ref.group_rows(off.cpu().numpy(), M)):
        ax, aw = np.abs(host(x)[a:b]), np.abs(host(w)[e])
        t = (2 * (k + 8) + 3) * U * (ax @ aw.T) + k * 2.0 ** -37 * ax.max(1)[:, None] * aw.max(1)[None]
        within(host(y)[a:b], ry[a:b], t + U * np.abs(ry[a:b]), f"group {e}")


# ---------------------------------------------------------------- orthogonalised update
def _growth(g, steps, coefficients=(3.4445, -4.7750, 2.0315)):
    """How much a relative error of each step's operands can grow until the result: a Frobenius
    perturbation passes a step multiplied by at most max|p'| over the singular values' range."""
    a, b, c = coefficients
    s = np.linalg.svd(g, compute_uv=False)
    s = s / np.sqrt((s ** 2).sum())
    norms, slopes = [], []
    for _ in range(steps):
        t = np.linspace(0, s.max() * 1.0001, 2001)
        norms.append(np.sqrt((s ** 2).sum()))
        slopes.append(np.abs(a + 3 * b * t ** 2 + 5 * c * t ** 4).max())
        s = a * s + b * s ** 3 + c * s ** 5
    norms.append(np.sqrt((s ** 2).sum()))
    total = 1.0
    for j in range(steps):
        total += np.prod(slopes[j:]) * norms[j] / norms[-1]
    return total


ORTHO = [(1, 1, 1), (1, 1, 5), (2, 7, 3), (3, 33, 64), (1, 64, 64), (2, 100, 131), (5, 128, 256),
         (2, 256, 96), (1, 320, 200), (1, 300, 517), (70, 40, 24)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,m,n", ORTHO)
def test_orthogonalize(B, m, n, dtype):
    r = np.random.default_rng(m * 1000 + n)
    x = dev(1e-3 * r.normal(size=(B, m, n)) * np.exp(r.normal(size=(1, 1, n))), dtype)
    say(f"orthogonalize B={B} m={m} n={n} {dtype}")
    out = mx.orthogonalize(x)
    torch.cuda.synchronize()
    for i in range(0, B, max(1, B // 5)):
        want = ref.orthogonalize(host(x[i]))
        # per step three products of at most max(m, n) terms with weights |a| + |b| + |c| < 11,
        # rounding like random signs: 2 u sqrt(K) each
        delta = 2 * U * 3 * 11 * np.sqrt(max(m, n))
        tol = delta * _growth(host(x[i]), 5) * np.linalg.norm(want)
        got = host(out[i])
        err = np.linalg.norm(got - want)
        assert err <= tol + (STORE[dtype] if dtype == "bf16" else 0) * np.linalg.norm(want), (i, err, tol)
        if dtype == "f32":  # and as exact as float32 products are
            plain = np.linalg.norm(ref.orthogonalize(host(x[i]), dtype=np.float32) - want)
            assert err <= 2 * plain + 1e-6 * np.linalg.norm(want), (i, err, plain)


@pytest.mark.parametrize("steps", [0, 1, 2])
def test_orthogonalize_steps_and_coefficients(steps):
    r = np.random.default_rng(steps)
    x = dev(r.normal(size=(3, 48, 80)))
    for coef in ((3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (15 / 8, -10 / 8, 3 / 8)):
        say(f"orthogonalize steps={steps} {coef}")
        out = mx.orthogonalize(x, steps=steps, eps=1e-3, coefficients=coef)
        torch.cuda.synchronize()
        for i in range(3):
            want = ref.orthogonalize(host(x[i]), steps, 1e-3, coef)
            tol = 2 * U * 33 * np.sqrt(80) * _growth(host(x[i]), steps, coef) * np.linalg.norm(want)
            assert np.linalg.norm(host(out[i]) - want) <= tol + 2 * U * np.linalg.norm(want)


def test_orthogonalize_zero_tiny_and_types():
    r = np.random.default_rng(8)
    g = r.normal(size=(3, 40, 56))
    g[1] = 0.0
    g[2] *= 1e-25                     # its squares leave float32's range
    x = dev(g)
    say("orthogonalize zero and tiny")
    out = mx.orthogonalize(x, eps=0.0)
    half = mx.orthogonalize(x, eps=0.0, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert not out[1].any()
    assert torch.equal(half, out.to(torch.bfloat16))
    want = ref.orthogonalize(host(x[2]), eps=0.0)
    assert np.linalg.norm(host(out[2]) - want) <= 1e-4 * np.linalg.norm(want)


def test_orthogonalize_blocks_of_a_weight_gradient_and_in_place():
    """The three matrices of every expert block, taken where layer_backward leaves them."""
    r = np.random.default_rng(9)
    N, d, I = 3, 64, 128
    dW = dev(r.normal(size=(N, 3, I * d)))
    before = dW.clone()
    down = dW[:, 2].view(N, d, I)
    say("orthogonalize strided")
    got = mx.orthogonalize(down)
    same = mx.orthogonalize(down.contiguous())
    torch.cuda.synchronize()
    assert torch.equal(got, same) and torch.equal(dW, before)
    assert mx.orthogonalize(down, out=down) is down
    torch.cuda.synchronize()
    assert torch.equal(down, same)
    assert torch.equal(dW[:, :2], before[:, :2])          # the other matrices are untouched
    out = torch.zeros(N, 3, I * d, device="cuda", dtype=torch.bfloat16)
    mx.orthogonalize(before[:, 0].view(N, I, d), out=out[:, 1].view(N, I, d))
    torch.cuda.synchronize()
    assert not out[:, 0].any() and not out[:, 2].any() and out[:, 1].any()


# ---------------------------------------------------------------- repeated, captured, other streams
def _calls():
    r = np.random.default_rng(12)
    x, w, b, dy = _norm_inputs(300, 256, "bf16", 3)
    _, mean, rstd = mx.layer_norm(x, w, b)
    gx, gw, off, gdy, _ = _grouped_inputs([100, 0, 33, 200], 0, 4, 192, 136, "f32", 4)
    hx, hw, hoff, hdy, _ = _grouped_inputs([100, 0, 33, 200], 0, 4, 192, 136, "bf16", 4)
    sx, sw, soff, _, _ = _grouped_inputs([2, 1, 3], 0, 0, 192, 128, "bf16", 4)
    g = dev(r.normal(size=(3, 96, 160)))
    return {
        "layer_norm": lambda: mx.layer_norm(x, w, b),
        "layer_norm_backward": lambda: mx.layer_norm_backward(dy, x, w, mean, rstd),
        "grouped_f32": lambda: (mx.grouped_matmul(gx, gw, off),),
        "grouped_bf16": lambda: (mx.grouped_matmul(hx, hw, hoff),),
        "grouped_few_rows": lambda: (mx.grouped_matmul(sx, sw, soff),),
        "grouped_backward_f32": lambda: mx.grouped_matmul_backward(gx, gw, off, gdy),
        "grouped_backward_bf16": lambda: mx.grouped_matmul_backward(hx, hw, hoff, hdy),
        "orthogonalize": lambda: (mx.orthogonalize(g),),
    }


CALLS = ["layer_norm", "layer_norm_backward", "grouped_f32", "grouped_bf16", "grouped_few_rows",
         "grouped_backward_f32", "grouped_backward_bf16", "orthogonalize"]


def _bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("name", CALLS)
def test_repeated_captured_and_on_another_stream(name):
    say(f"repeat {name}")
    call = _calls()[name]
    want = call()
    torch.cuda.synchronize()
    say(f"other stream {name}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(_bits(a), _bits(b))
    say(f"capture {name}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call()
    for k in range(3):
        for t in captured:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(_bits(a), _bits(b)), f"replay {k}"
        again = call()                       # eager work between the replays
        torch.cuda.synchronize()
        for a, b in zip(again, want):
            assert torch.equal(_bits(a), _bits(b))


# ---------------------------------------------------------------- a step of a block, as used together
def test_a_training_step_of_a_block_with_experts_of_its_own():
    """Norm, routing, ReLU experts out of grouped products, their gradients and the
    orthogonalised update, against the same step in float64 with the routing held fixed."""
    torch.manual_seed(0)
    T, d, I, N, K = 96, 128, 192, 8, 2
    f = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    x, nw, nb, E = f(T, d), 1 + 0.1 * f(d), 0.1 * f(d), 0.3 * f(N, d)
    w1, w2 = 0.1 * f(N, I, d), 0.1 * f(N, d, I)
    say("block step")
    u, mean, rstd = mx.layer_norm(x, nw, nb)
    idx, gate, _ = mx.route(u, E, K)
    _, off, pair = mx.dispatch(idx, N)
    tok = (pair // K).long()
    g = gate.view(-1)[pair.long()][:, None]
    xs = u[tok].contiguous()
    h = mx.grouped_matmul(xs, w1, off)
    a = h.clamp(min=0)
    y = mx.grouped_matmul(a, w2, off)
    dout = f(T, d)                                   # gradient of the step's output
    dy = (dout[tok] * g).contiguous()
    da, dw2 = mx.grouped_matmul_backward(a, w2, off, dy)
    dxs, dw1 = mx.grouped_matmul_backward(xs, w1, off, (da * (h > 0)).contiguous())
    du = torch.zeros_like(u).index_add_(0, tok, dxs)
    dx, dnw, dnb = mx.layer_norm_backward(du, x, nw, mean, rstd)
    step1 = mx.orthogonalize(dw1)
    torch.cuda.synchronize()

    offh, tokh, gh = off.cpu().numpy(), tok.cpu().numpy(), host(g)
    ru, rmean, rrstd = ref.layer_norm(host(x), host(nw), host(nb), 1e-5)
    rh, _ = ref.grouped_matmul(ru[tokh], host(w1), offh)
    ra = np.maximum(rh, 0)
    ry, _ = ref.grouped_matmul(ra, host(w2), offh)
    rdy = host(dout)[tokh] * gh
    rda, rdw2 = ref.grouped_matmul_backward(ra, host(w2), offh, rdy)
    rdxs, rdw1 = ref.grouped_matmul_backward(ru[tokh], host(w1), offh, rda * (rh > 0))
    rdu = np.zeros_like(ru)
    np.add.at(rdu, tokh, rdxs)
    rdx, rdnw, rdnb = ref.layer_norm_backward(rdu, host(x), host(nw), rmean, rrstd)
    # chains of at most five sums of up to 192 terms: 5 * 200 * 2 u = 1.2e-4 of the largest
    for got, want, label in ((y, ry, "y"), (dw2, rdw2, "dw2"), (dw1, rdw1, "dw1"), (dx, rdx, "dx"),
                             (dnw, rdnw, "dnw"), (dnb, rdnb, "dnb")):
        within(got, want, 1.2e-4 * np.abs(want).max(), label)
    counts = np.diff(offh)
    for e in range(N):
        if counts[e] >= 1:
            want = ref.orthogonalize(host(dw1[e]))
            assert np.linalg.norm(host(step1[e]) - want) <= 1e-3 * np.linalg.norm(want)
