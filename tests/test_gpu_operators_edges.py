"""The operators beside the layer where they can go wrong: infinities and NaN among the
operands, tensors past 2^32 bytes, workspaces shared by captured graphs, empty batches, and
the orthogonalised update on both sides of its size rule.  Tolerances are those of
test_gpu_operators.py."""
import numpy as np
import pytest
import torch

from oracle import operators as ref
from parity_helpers import say
from test_gpu_operators import (STORE, U, _bits, _grouped_inputs, _growth, _offsets, _sum_tol, dev,
                                host, mx, within)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- values that are not finite
def _same_where_finite(got, want, tol, label):
    """got is not finite exactly where want is not, and within tol elsewhere."""
    g = host(got)
    assert (np.isfinite(g) == np.isfinite(want)).all(), label
    ok = np.isfinite(want)
    within(np.where(ok, g, 0.0), np.where(ok, want, 0.0), np.where(ok, tol, 1.0), label)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,k", [(48, 72), (320, 256)])
def test_grouped_bad_values_reach_their_own_results_only(n, k, dtype):
    sizes = [30, 150, 0, 9]
    x, w, off, dy, _ = _grouped_inputs(sizes, 2, 3, n, k, dtype, 21)
    x[2 + 5, 7] = float("inf")
    x[2 + 31, 0] = float("nan")
    w[1, 3, 11] = -float("inf")
    w[3, n - 1, k - 1] = float("nan")
    dy[2 + 40, 6] = float("inf")
    dy[2 + 182] = float("nan")               # a whole row
    say(f"grouped bad values n={n} k={k} {dtype}")
    y = mx.grouped_matmul(x, w, off)
    dx, dw = mx.grouped_matmul_backward(x, w, off, dy)
    torch.cuda.synchronize()
    offs = off.cpu().numpy()
    fx, fw, fdy = (np.where(np.isfinite(host(t)), np.abs(host(t)), 0.0) for t in (x, w, dy))
    most = fx[2:191].max() * fdy[2:191].max()
    with np.errstate(invalid="ignore"):
        for e, (a, b) in enumerate(ref.group_rows(offs, x.shape[0])):
            X, W, DY = host(x)[a:b], host(w)[e], host(dy)[a:b]
            t = _sum_tol(fx[a:b], fw[e], k, dtype)
            want = X @ W.T
            _same_where_finite(y[a:b], want, t + STORE[dtype] * (np.abs(want) + t), f"y {e}")
            t = _sum_tol(fdy[a:b], fw[e].T, n, dtype)
            want = DY @ W
            _same_where_finite(dx[a:b], want, t + STORE[dtype] * (np.abs(want) + t), f"dx {e}")
            t = _sum_tol(fdy[a:b].T, fx[a:b].T, b - a, dtype)
            t = t + (b - a) * 2.0 ** -37 * most * (dtype == "f32")
            want = DY.T @ X
            _same_where_finite(dw[e], want, t + U * np.abs(want), f"dw {e}")


@pytest.mark.parametrize("steps", [0, 1, 5])
@pytest.mark.parametrize("m,n", [(33, 64), (96, 100), (200, 300)])
def test_orthogonalize_keeps_a_bad_matrix_to_itself(m, n, steps):
    r = np.random.default_rng(22)
    x = dev(r.normal(size=(4, m, n)))
    clean = mx.orthogonalize(x, steps=steps)
    x[1, 2, 3] = float("nan")
    x[3, m - 1, n - 1] = float("inf")
    say(f"orthogonalize bad values {m}x{n}")
    out = mx.orthogonalize(x, steps=steps)
    torch.cuda.synchronize()
    for i in (0, 2):
        assert torch.equal(_bits(out[i]), _bits(clean[i]))
    assert torch.isnan(out[1]).all()
    if steps:                                 # (without steps a / inf is a zero)
        assert torch.isnan(out[3]).all()
    else:
        assert torch.isnan(out[3, m - 1, n - 1]) and not out[3].nan_to_num().any()


def test_layer_norm_backward_of_an_empty_batch():
    for dt in (torch.float32, torch.bfloat16):
        for d in (5, 512, 20000):
            say(f"layer_norm T=0 d={d}")
            x = torch.empty(0, d, device="cuda", dtype=dt)
            w = torch.ones(d, device="cuda", dtype=dt)
            y, mean, rstd = mx.layer_norm(x, w)
            dx, dw, db = mx.layer_norm_backward(x, x, w, mean, rstd)
            torch.cuda.synchronize()
            assert y.shape == dx.shape == (0, d) and mean.shape == rstd.shape == (0,)
            assert dw.shape == db.shape == (d,) and not dw.any() and not db.any()


def test_grouped_empty_batch_one_gradient_only():
    for dt in (torch.float32, torch.bfloat16):
        say(f"grouped M = 0 {dt}")
        w = torch.randn(3, 32, 200, device="cuda").to(dt)
        off = torch.zeros(4, dtype=torch.int32, device="cuda")
        x, dy = torch.empty(0, 200, device="cuda", dtype=dt), torch.empty(0, 32, device="cuda", dtype=dt)
        dx, none = mx.grouped_matmul_backward(x, w, off, dy, need_dw=False)
        assert dx.shape == (0, 200) and none is None
        none, dw = mx.grouped_matmul_backward(x, w, off, dy, need_dx=False)
        torch.cuda.synchronize()
        assert none is None and dw.shape == w.shape and not dw.any()


# ---------------------------------------------------------------- the update's two paths
# (batches and sides around 64, 128 and the rule's limits; tall and wide; odd sizes)
PATHS = [(1, 1, 300), (2, 64, 65), (1, 65, 65), (3, 63, 449), (1, 64, 513), (1, 513, 64), (2, 128, 129),
         (2, 129, 128), (1, 128, 257), (3, 129, 131), (127, 20, 2500), (128, 20, 2500), (17, 128, 1000),
         (130, 130, 65), (140, 100, 700), (300, 9, 10), (2, 500, 130), (1, 1100, 700)]


def _check_update(got, g, steps, coef, dtype, label):
    want = ref.orthogonalize(g, steps, 1e-7, coef)
    delta = 2 * U * 3 * 11 * np.sqrt(max(g.shape))
    tol = (delta * _growth(g, steps, coef) + 2 * U + (STORE["bf16"] if dtype == "bf16" else 0))
    err = np.linalg.norm(host(got) - want)
    assert err <= tol * np.linalg.norm(want), (label, err, tol * np.linalg.norm(want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,m,n", PATHS)
def test_orthogonalize_both_paths(B, m, n, dtype):
    r = np.random.default_rng(B + 1000 * m + n)
    x = dev(r.normal(size=(B, m, n)) * 10.0 ** r.uniform(-6, 6, (B, 1, 1)), dtype)
    usual = (3.4445, -4.7750, 2.0315)
    for steps, coef in ((5, usual), (1, usual), (3, (1.5, -0.5, 0.0))):
        say(f"orthogonalize B={B} {m}x{n} {dtype} steps={steps}")
        out = mx.orthogonalize(x, steps=steps, coefficients=coef)
        again = mx.orthogonalize(x, steps=steps, coefficients=coef)
        torch.cuda.synchronize()
        assert torch.equal(_bits(out), _bits(again))
        for i in sorted({0, B // 2, B - 1}):
            _check_update(out[i], host(x[i]), steps, coef, dtype, (i, steps))
    mine = x.clone()
    assert mx.orthogonalize(mine, out=mine) is mine
    want = mx.orthogonalize(x)
    other = mx.orthogonalize(x, out_dtype=torch.float32 if dtype == "bf16" else torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(_bits(mine), _bits(want))
    low = (other if dtype == "f32" else want)
    assert torch.equal(_bits(low), _bits((want if dtype == "f32" else other).to(torch.bfloat16)))


# ---------------------------------------------------------------- past 2^32 bytes
def _rows_match(got, want, a, b, n, dtype, label):
    t = _sum_tol(np.abs(a), np.abs(b), n, dtype)
    within(got, want, t + STORE[dtype] * (np.abs(want) + t), label)


def test_grouped_rows_past_4_gib():
    M, k, n, E = 300_001, 8192, 24, 3
    torch.manual_seed(1)
    x = torch.randn(M, k, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(E, n, k, device="cuda", dtype=torch.bfloat16)
    off = torch.tensor([0, 100, 299_990, 300_000], dtype=torch.int32, device="cuda")
    say("grouped x of 4.9 GB")
    y = mx.grouped_matmul(x, w, off)
    dy = torch.randn(M, n, device="cuda", dtype=torch.bfloat16)
    dx, _ = mx.grouped_matmul_backward(x, w, off, dy, need_dw=False)
    torch.cuda.synchronize()
    for e, (a, b) in enumerate([(0, 100), (299_900, 299_990), (299_990, 300_000)]):
        X, W, DY = host(x[a:b]), host(w[e]), host(dy[a:b])
        _rows_match(y[a:b], X @ W.T, X, W, k, "bf16", f"y {e}")
        _rows_match(dx[a:b], DY @ W, DY, W.T, n, "bf16", f"dx {e}")
    assert not y[-1].any() and not dx[-1].any()


def test_grouped_weights_and_their_gradient_past_4_gib():
    E, n, k = 600, 1024, 2048
    torch.manual_seed(2)
    sizes = np.zeros(E, int)
    sizes[[0, 300, 598, 599]] = 3, 70, 1, 6
    M = int(sizes.sum())
    x = torch.randn(M, k, device="cuda")
    w = torch.randn(E, n, k, device="cuda")
    dy = torch.randn(M, n, device="cuda")
    off = torch.from_numpy(_offsets(sizes)).cuda()
    say("grouped w of 5 GB")
    y = mx.grouped_matmul(x, w, off)
    dx, dw = mx.grouped_matmul_backward(x, w, off, dy)
    torch.cuda.synchronize()
    most = np.abs(host(x)).max() * np.abs(host(dy)).max()
    for e, (a, b) in enumerate(ref.group_rows(off.cpu().numpy(), M)):
        if a == b:
            continue
        X, W, DY = host(x[a:b]), host(w[e]), host(dy[a:b])
        _rows_match(y[a:b], X @ W.T, X, W, k, "f32", f"y {e}")
        _rows_match(dx[a:b], DY @ W, DY, W.T, n, "f32", f"dx {e}")
        t = _sum_tol(np.abs(DY).T, np.abs(X).T, b - a, "f32") + (b - a) * 2.0 ** -37 * most
        within(dw[e], DY.T @ X, t + U * np.abs(DY.T @ X), f"dw {e}")
    assert not dw[1:300].any() and not dw[301:598].any()


def test_layer_norm_past_4_gib():
    T, d = 600_003, 4096
    torch.manual_seed(3)
    x = torch.randn(T, d, device="cuda", dtype=torch.bfloat16)
    say("layer_norm of 4.9 GB")
    y, mean, rstd = mx.layer_norm(x)
    dx, _, _ = mx.layer_norm_backward(x, x, None, mean, rstd)
    torch.cuda.synchronize()
    for rows in (slice(0, 4), slice(T - 4, T)):
        small, m, s = mx.layer_norm(x[rows].clone())
        again = mx.layer_norm_backward(x[rows].clone(), x[rows].clone(), None, m, s)[0]
        torch.cuda.synchronize()
        assert torch.equal(_bits(y[rows]), _bits(small)) and torch.equal(mean[rows], m)
        assert torch.equal(rstd[rows], s) and torch.equal(_bits(dx[rows]), _bits(again))


# ---------------------------------------------------------------- the widest rows
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,k", [(100, 1 << 20), (1 << 20, 100), (96, (1 << 20) - 1), (1, 1 << 20)])
def test_grouped_widest_rows(n, k, dtype):
    """n and k up to 2^20, against the definition in float64 on the GPU (one group and a rest)."""
    M, a, b = 300, 7, 297
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    torch.manual_seed(7)
    x, w = torch.randn(M, k, device="cuda").to(dt), torch.randn(1, n, k, device="cuda").to(dt)
    dy = torch.randn(M, n, device="cuda").to(dt)
    off = torch.tensor([a, b], dtype=torch.int32, device="cuda")
    say(f"grouped n={n} k={k} {dtype}")
    y = mx.grouped_matmul(x, w, off)
    dx, dw = mx.grouped_matmul_backward(x, w, off, dy)
    torch.cuda.synchronize()
    X, W, DY = x[a:b].double(), w[0].double(), dy[a:b].double()

    def check(got, p, q, terms, store, label):
        """got = p q within the bounds of test_gpu_grouped_float32.py."""
        want, t = p @ q, (12 * (terms + 8) + 8) * U * (p.abs() @ q.abs())
        if dtype == "f32" and label == "y":
            t += 2.0 ** -37.9 * (p.abs().amax(1)[:, None] * q.abs().sum(0) +
                                 p.abs().sum(1)[:, None] * q.abs().amax(0))
        assert _every_row(got, want, t + store * (want.abs() + t)), label

    check(y[a:b], X, W.t().contiguous(), k, STORE[dtype], "y")
    check(dx[a:b], DY, W, n, STORE[dtype], "dx")
    check(dw[0], DY.t().contiguous(), X, b - a, U, "dw")
    for t in (y, dx):
        assert not t[:a].any() and not t[b:].any()


# ---------------------------------------------------------------- past 2^26 rows
# (a launch of one wavefront per row would hold 2^32 threads, of which some would never run)
def _every_row(got, want, tol):
    """On the GPU: |got - want| <= tol for every element (float64 tensors)."""
    return bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grouped_past_2_26_rows(dtype):
    M, n, k = (1 << 26) + 5, 8, 24
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    torch.manual_seed(4)
    x = torch.randn(M, k, device="cuda").to(dt)
    w = torch.randn(2, n, k, device="cuda").to(dt)
    off = torch.tensor([1, M - 1000, M - 2], dtype=torch.int32, device="cuda")
    say(f"grouped y of 2^26 rows {dtype}")
    y = mx.grouped_matmul(x, w, off)
    torch.cuda.synchronize()
    for a in range(0, M, 1 << 24):
        b = min(M, a + (1 << 24))
        e = (torch.arange(a, b, device="cuda") >= M - 1000).long()
        want = torch.zeros(b - a, n, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(want)
        for g in (0, 1):
            X, W = x[a:b].double(), w[g].double()
            want += (X @ W.t().contiguous()) * (e == g)[:, None]
            size += (X.abs() @ W.abs().t().contiguous()) * (e == g)[:, None]
        t = (2 * (k + 8) + 8) * U * size
        if a == 0:
            want[0], t[0] = 0, 0
        if b == M:
            want[-2:], t[-2:] = 0, 0
        assert _every_row(y[a:b], want, t + STORE[dtype] * (want.abs() + t)), a
    del y
    dy = torch.randn(M, n, device="cuda").to(dt)
    off = torch.tensor([M - 900, M - 300, M - 2], dtype=torch.int32, device="cuda")
    say(f"grouped gradients of 2^26 rows {dtype}")
    dx, dw = mx.grouped_matmul_backward(x, w, off, dy)
    torch.cuda.synchronize()
    assert not dx[:M - 900].any() and not dx[M - 2:].any()
    for e, (a, b) in enumerate([(M - 900, M - 300), (M - 300, M - 2)]):
        X, W, DY = host(x[a:b]), host(w[e]), host(dy[a:b])
        t = (12 * (n + 8) + 8) * U * (np.abs(DY) @ np.abs(W))
        within(dx[a:b], DY @ W, t + STORE[dtype] * (np.abs(DY @ W) + t), f"dx {e}")
        t = (12 * (b - a + 8) + 8) * U * (np.abs(DY).T @ np.abs(X))
        within(dw[e], DY.T @ X, t + U * np.abs(DY.T @ X), f"dw {e}")


def test_grouped_past_2_26_weight_rows():
    """As many rows of w: E * n."""
    E, n, k, M = 1024, 1 << 16, 8, 40
    torch.manual_seed(5)
    w = torch.randn(E, n, k, device="cuda", dtype=torch.bfloat16)
    w = torch.cat([w, w[:, :128]], 1).contiguous()
    x = torch.randn(M, k, device="cuda", dtype=torch.bfloat16)
    sizes = np.zeros(E, int)
    sizes[[0, 500, 1023]] = 30, 1, 9
    off = torch.from_numpy(_offsets(sizes)).cuda()
    say("grouped y with 2^26 rows of w")
    y = mx.grouped_matmul(x, w, off)
    torch.cuda.synchronize()
    for e, (a, b) in enumerate(ref.group_rows(off.cpu().numpy(), M)):
        if a < b:
            X, W = host(x[a:b]), host(w[e])
            _rows_match(y[a:b], X @ W.T, X, W, k, "bf16", f"y {e}")


def test_orthogonalize_past_2_26_rows():
    torch.manual_seed(6)
    x = torch.randn(65535, 1100, 1, device="cuda")
    say("orthogonalize of 72e6 rows, no steps")
    out = mx.orthogonalize(x, steps=0)
    want = x.double() / (x.double().square().sum((1, 2), keepdim=True).sqrt() + 1e-7)
    assert _every_row(out, want, 2 * U * want.abs())
    del x, out, want
    x = torch.randn(64, 1 << 20, 1, device="cuda")
    say("orthogonalize of 2^26 rows")
    out = mx.orthogonalize(x)
    torch.cuda.synchronize()
    for i in (0, 63):
        _check_update(out[i], host(x[i]), 5, (3.4445, -4.7750, 2.0315), "f32", i)


# ---------------------------------------------------------------- captured graphs
def test_graphs_that_share_a_workspace():
    """Every operator that needs one, captured into graphs of its own over one workspace and
    replayed in turn, with eager calls on the same workspace between."""
    r = np.random.default_rng(31)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    gx, gw, off, gdy, _ = _grouped_inputs([100, 0, 33, 200], 0, 4, 192, 136, "f32", 4)
    hx, hw, hoff, hdy, _ = _grouped_inputs([64, 7, 300], 1, 0, 200, 150, "bf16", 5)
    x, w = dev(r.normal(size=(300, 256)), "bf16"), dev(r.normal(size=256), "bf16")
    _, mean, rstd = mx.layer_norm(x, w)
    small, large = dev(r.normal(size=(3, 96, 160))), dev(r.normal(size=(2, 700, 600)))
    calls = [
        lambda: (mx.grouped_matmul(gx, gw, off, workspace=ws),),
        lambda: mx.grouped_matmul_backward(gx, gw, off, gdy, workspace=ws),
        lambda: (mx.grouped_matmul(hx, hw, hoff, workspace=ws),),
        lambda: mx.grouped_matmul_backward(hx, hw, hoff, hdy, workspace=ws),
        lambda: mx.layer_norm_backward(x, x, w, mean, rstd, workspace=ws),
        lambda: (mx.orthogonalize(small, workspace=ws),),
        lambda: (mx.orthogonalize(large, workspace=ws),),
    ]
    want = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i, c in enumerate(calls):
        say(f"capture {i}")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    for k in range(3):
        ws.fill_(255)                        # what other calls left there does not matter
        for i in ((0, 1, 2, 3, 4, 5, 6), (6, 0, 5, 2, 4, 1, 3), (3, 3, 6, 6, 1, 0, 5))[k]:
            say(f"replay {k} {i}")
            for t in outs[i]:
                t.zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            for a, b in zip(outs[i], want[i]):
                assert torch.equal(_bits(a), _bits(b)), (k, i)
            for a, b in zip(calls[i](), want[i]):
                assert torch.equal(_bits(a), _bits(b)), (k, i)


# ---------------------------------------------------------------- float32 products of few rows
FEW = [([1], 0, 0, 32, 4), ([2, 0, 1], 1, 2, 33, 8), ([33, 0, 0, 1, 64, 65, 0, 3], 0, 4, 70, 36),
       ([150] + [0] * 7, 0, 0, 129, 100), ([1] * 64, 0, 0, 64, 1000), ([31, 32, 33, 64, 96], 3, 0, 260, 516),
       ([64] * 3, 0, 0, 96, 2052), ([64] * 3 + [1], 0, 1, 31, 2052), ([5, 9], 0, 0, 200, 30),
       ([0, 0, 7, 0], 2, 1, 1408, 2048), ([3] * 200 + [0] * 300, 5, 5, 40, 68)]


@pytest.mark.parametrize("case", range(len(FEW)))
def test_grouped_f32_few_rows(case):
    from test_gpu_operators import _grouped_check
    _grouped_check(*FEW[case], "f32", seed=100 + case)


def test_grouped_f32_few_rows_at_the_ends_of_the_range():
    """Weights and rows near float32's largest and smallest values: no product leaves the
    range on the way to a result inside it."""
    r = np.random.default_rng(41)
    M, E, n, k = 12, 3, 64, 128
    x, w = r.normal(size=(M, k)), r.normal(size=(E, n, k))
    x[0] *= 1e-36
    w[0, 0] = 3e38 * np.sign(w[0, 0])          # sums of 128 such products with a small row
    w[1] *= 1e-28
    x[5] *= 1e30
    w[2, 3] = 0.0
    x[11] = 0.0
    x, w = dev(x), dev(w)
    off = torch.tensor([0, 1, 8, 12], dtype=torch.int32, device="cuda")
    say("grouped f32 few rows, ends of the range")
    y = mx.grouped_matmul(x, w, off)
    torch.cuda.synchronize()
    ry, _ = ref.grouped_matmul(host(x), host(w), off.cpu().numpy())
    for e, (a, b) in enumerate([(0, 1), (1, 8), (8, 12)]):
        ax, aw = np.abs(host(x)[a:b]), np.abs(host(w)[e])
        t = (2 * (k + 8) + 3) * U * (ax @ aw.T)
        within(y[a:b], ry[a:b], t + U * np.abs(ry[a:b]), f"group {e}")


# (rows of one group past a tile, widths past a k-step and a tile, both gradients and dx alone)
FEW_DX = [([1], 0, 0, 32, 192), ([2, 0, 1], 1, 2, 36, 196), ([33, 0, 0, 1, 64, 65, 0, 3], 0, 4, 100, 260),
          ([150] + [0] * 7, 0, 0, 132, 708), ([3] * 200 + [0] * 300, 5, 5, 40, 192), ([64] * 3, 0, 0, 96, 2052),
          ([64] * 3 + [1], 0, 1, 96, 2052), ([0, 0, 7, 0], 2, 1, 1408, 2048)]


@pytest.mark.parametrize("case", range(len(FEW_DX)))
def test_grouped_f32_few_rows_gradients(case):
    from test_gpu_operators import _grouped_check
    sizes, before, behind, n, k = FEW_DX[case]
    _grouped_check(sizes, before, behind, n, k, "f32", seed=200 + case)
    x, w, off, dy, _ = _grouped_inputs(sizes, before, behind, n, k, "f32", 200 + case)
    both = mx.grouped_matmul_backward(x, w, off, dy)
    dx, _ = mx.grouped_matmul_backward(x, w, off, dy, need_dw=False)
    _, dw = mx.grouped_matmul_backward(x, w, off, dy, need_dx=False)
    torch.cuda.synchronize()
    assert torch.equal(_bits(dx), _bits(both[0])) and torch.equal(_bits(dw), _bits(both[1]))


def test_grouped_f32_few_rows_gradient_keeps_bad_weights_to_their_columns():
    x, w, off, dy, _ = _grouped_inputs([9, 40], 0, 0, 44, 200, "f32", 51)
    clean = mx.grouped_matmul_backward(x, w, off, dy, need_dw=False)[0]
    w[0, 43, 7] = float("inf")               # the last row, which padding must not reach
    w[1, 0, 199] = float("nan")
    dx = mx.grouped_matmul_backward(x, w, off, dy, need_dw=False)[0]
    torch.cuda.synchronize()
    bad = torch.zeros_like(dx, dtype=torch.bool)
    bad[:9, 7] = True
    bad[9:, 199] = True
    assert (~torch.isfinite(dx) == bad).all() and torch.equal(dx[~bad], clean[~bad])


@pytest.mark.parametrize("m,n", [(8, 16), (20, 30), (30, 500), (64, 64), (64, 700), (100, 120), (128, 256)])
def test_orthogonalize_small_matrices_are_as_exact_as_float32_products(m, n):
    """Root mean square over 16 matrices of the error against 64 bits: at most twice that of the
    same steps in float32 (operands of 22 bits and more against 24, sums of the same length)."""
    r = np.random.default_rng(m + n)
    x = dev(r.normal(size=(16, m, n)))
    out = mx.orthogonalize(x)
    torch.cuda.synchronize()
    own, plain = [], []
    for i in range(16):
        want = ref.orthogonalize(host(x[i]))
        own.append(np.linalg.norm(host(out[i]) - want))
        plain.append(np.linalg.norm(ref.orthogonalize(host(x[i]), dtype=np.float32) - want))
    assert np.square(own).sum() <= 4 * np.square(plain).sum(), (own, plain)


@pytest.mark.parametrize("m,n", [(128, 1500), (64, 2100), (700, 100)])
def test_orthogonalize_many_matrices_repeat_their_bits(m, n):
    """One block per matrix on every CU, iterates past the caches: what a chunk's loads and the
    stores of another do to each other shows as bits that change from call to call."""
    torch.manual_seed(61)
    x = torch.randn(512, m, n, device="cuda")
    want = mx.orthogonalize(x)
    for k in range(4):
        say(f"orthogonalize 512 x {m} x {n}, call {k}")
        got = mx.orthogonalize(x)
        torch.cuda.synchronize()
        assert torch.equal(_bits(got), _bits(want)), k
    for i in (0, 255, 511):
        _check_update(want[i], host(x[i]), 5, (3.4445, -4.7750, 2.0315), "f32", i)
