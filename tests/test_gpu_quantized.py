"""GPU parity of the RMS norm, the 8-bit operators and the balance loss against their float64
oracle.

Tolerances, per element, u = 2^-24:
  sums     a row's sum of squares goes through at most 64 additions in a thread and 26 across
           threads, each square rounded once: 96 u; rstd halves that, its root and quotient
           add 4 u; a sum of n products of 8-bit values (exact products) is off by at most
           (n + 8) 2 u sum|products| in any order, each addition by at most one unit (2 u)
           whatever way the matrix instructions round, and each block's scale (a product of
           two) by 4 u more;
  cut      bfloat16 results of 8-bit products come from sums of eight neighbours, in an order of
           the contraction that is the kernel's own, each product cut off below 2^-13 of the
           largest of the eight: at most 7 products of eight lose at most 2^-13 of the largest
           each, so a block of 128 loses at most 16 * 7 * 2^-13 = 2^-6.2 of its largest product;
           and 2^-10 of the sum of |products|, as the largest of eight is at most their sum;
  store    half a step of the stored type, relative: 2^-8 for bfloat16, u for float32;
  8 bits   q is the rounding of some value within the error of what is rounded, so it lies
           between the roundings of both ends of that interval (rounding is monotone); dividing
           by a scale costs 4 u (the scale's rounding, its reciprocal's, the product's).
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
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
STORE = {"f32": U, "bf16": 2.0 ** -8}
LEAST = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134}    # half a step of the smallest numbers


def dev(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to("cuda").to(DT[dtype])


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def host(t):
    return t.double().cpu().numpy()


def within(got, want, tol, label):
    err = np.abs(host(got) - want) if torch.is_tensor(got) else np.abs(got - want)
    bad = ~(err <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err / np.maximum(tol, 1e-300), 0)), err.shape)
        raise AssertionError(f"{label}: {bad.sum()} of {bad.size} beyond tolerance, worst at {i}: "
                             f"error {err[i]:.3e}, tolerance {np.broadcast_to(tol, err.shape)[i]:.3e}")


def rounded(q, v, rel, kind, label):
    """q is the 8-bit rounding of a value within rel of v, relatively; NaN where v is not finite."""
    q = host(q)
    fine = np.isfinite(v)
    assert np.isnan(q[~fine]).all() and not np.isnan(q[fine]).any(), label
    lo, hi = v * (1 - np.sign(v) * rel), v * (1 + np.sign(v) * rel)
    most = ref.F8[kind][2]
    lo, hi = (ref.round_f8(np.clip(np.where(fine, x, 0), -most, most), kind) for x in (lo, hi))
    bad = fine & ~((lo <= q) & (q <= hi))
    assert not bad.any(), f"{label}: {bad.sum()} of {bad.size} are not the rounding, first {np.argwhere(bad)[0]}"


# ---------------------------------------------------------------- RMS norm
NORM_SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 64), (2, 513), (4, 512), (7, 1000), (33, 1024),
               (9, 1283), (6, 2050), (5, 4096), (3, 5001), (2, 8192), (3, 16400), (2, 20000),
               (1, 70001), (700, 72), (2051, 130), (9000, 16)]
RSTD = 48 * U + 4 * U      # relative error of rstd (see above)


def _norm_inputs(T, d, dtype, seed):
    r = np.random.default_rng(seed)
    x = dev(r.normal(size=(T, d)) * (1 + 3 * r.random((T, 1))) * np.exp(r.normal(size=d)), dtype)
    res = dev(2 * r.normal(size=(T, d)), dtype)
    w = dev(1 + 0.3 * r.normal(size=d), dtype)
    return x, res, w, dev(r.normal(size=(T, d)), dtype), dev(r.normal(size=(T, d)), dtype)


def _stream_check(x, res, h, dtype, label):
    want = host(x) if res is None else host((x.float() + res.float()).to(x.dtype))
    assert np.array_equal(host(h), want), label + " h"      # one rounding: the same bits
    return want


def _norm_check(x, w, res, eps, dtype, label):
    y, h, rstd = mx.rms_norm(x, w, res, eps)
    torch.cuda.synchronize()
    hh = _stream_check(x, res, h, dtype, label)
    ry, rr = ref.rms_norm(hh, None if w is None else host(w), eps)
    within(rstd, rr, RSTD * rr, label + " rstd")
    tol = (RSTD + 3 * U) * np.abs(ry)
    within(y, ry, tol + STORE[dtype] * (np.abs(ry) + tol), label + " y")
    return h, rstd


def _norm_f8_check(x, w, res, eps, dtype, kind, label):
    q, scales, h, rstd = mx.rms_norm_quantized(x, w, res, eps, F8[kind])
    torch.cuda.synchronize()
    assert q.dtype == F8[kind] and q.shape == x.shape
    hh = _stream_check(x, res, h, dtype, label)
    ry, rr = ref.rms_norm(hh, None if w is None else host(w), eps)
    within(rstd, rr, RSTD * rr, label + " rstd")
    rs = ref.block_scales(ry, kind)
    rel = RSTD + 3 * U
    within(scales, rs, (rel + U) * rs, label + " scales")
    # the value and the scale it is divided by both carry the row's error
    rounded(q, ry / ref.spread_rows(rs, x.shape[1]), 2 * rel + 4 * U, kind, label + " q")


def _norm_backward_check(dy, h, w, rstd, dh, dtype, label):
    dx, dw = mx.rms_norm_backward(dy, h, w, rstd, dh)
    torch.cuda.synchronize()
    g = host(dy) if w is None else host(dy) * host(w)
    rs = host(rstd)[:, None]
    hh = host(h) * rs
    rdx, rdw = ref.rms_norm_backward(host(dy), host(h), None if w is None else host(w), host(rstd),
                                     None if dh is None else host(dh))
    # mean(g hh): its products carry 3 u, its sum 96 u
    e2 = 100 * U * np.abs(g * hh).mean(1, keepdims=True)
    tol = rs * (np.abs(hh) * e2 + 6 * U * (np.abs(g) + np.abs(hh) * np.abs((g * hh).mean(1, keepdims=True))))
    tol = tol + 2 * U * np.abs(rdx) + (0 if dh is None else U * np.abs(host(dh)))
    within(dx, rdx, tol + STORE[dtype] * (np.abs(rdx) + tol), label + " dx")
    within(dw, rdw, (h.shape[0] + 12) * U * np.abs(host(dy) * hh).sum(0), label + " dweight")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", NORM_SHAPES)
def test_rms_norm(T, d, dtype):
    say(f"rms_norm T={T} d={d} {dtype}")
    x, res, w, dy, dh = _norm_inputs(T, d, dtype, T * 31 + d)
    h, rstd = _norm_check(x, w, res, 1e-6, dtype, "residual")
    _norm_check(x, None, None, 1e-2, dtype, "plain")
    _norm_backward_check(dy, h, w, rstd, dh, dtype, "residual")
    _norm_backward_check(dy, h, None, rstd, None, dtype, "plain")


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", NORM_SHAPES)
def test_rms_norm_quantized(T, d, dtype, kind):
    say(f"rms_norm_quantized T={T} d={d} {dtype} {kind}")
    x, res, w, _, _ = _norm_inputs(T, d, dtype, T * 37 + d)
    _norm_f8_check(x, w, res, 1e-6, dtype, kind, "residual")
    _norm_f8_check(x, None, None, 1e-2, dtype, kind, "plain")


def test_rms_norm_in_place_and_empty():
    say("rms_norm in place")
    for d in (96, 20000):
        x, res, w, dy, dh = _norm_inputs(5, d, "bf16", d)
        y, h, rstd = mx.rms_norm(x, w, res)
        for into in ("x", "res"):
            a, b = x.clone(), res.clone()
            t = a if into == "x" else b
            y2, h2, _ = mx.rms_norm(a, w, b, h_out=t)
            assert h2 is t and torch.equal(t, h) and torch.equal(y2, y)
            assert torch.equal(b if into == "x" else a, res if into == "x" else x)
        a = x.clone()
        assert torch.equal(mx.rms_norm(a, w, None, h_out=a)[0], mx.rms_norm(x, w)[0])
        assert torch.equal(a, x)
        dx, dw = mx.rms_norm_backward(dy, h, w, rstd, dh)
        g = dh.clone()
        dx2, dw2 = mx.rms_norm_backward(dy, h, w, rstd, g, out=g)
        assert dx2 is g and torch.equal(g, dx) and torch.equal(dw2, dw)
    e = torch.empty(0, 64, device="cuda")
    y, h, rstd = mx.rms_norm(e, None, e)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    q, s, _, _ = mx.rms_norm_quantized(e)
    assert q.shape == (0, 64) and s.shape == (0, 1)
    dx, dw = mx.rms_norm_backward(e, e, None, rstd)
    assert not dw.any() and dw.shape == (64,)


def test_rms_norm_keeps_a_bad_row_to_itself():
    r = np.random.default_rng(2)
    a = r.normal(size=(6, 256))
    clean = mx.rms_norm(dev(a))[0]
    q0, s0, _, _ = mx.rms_norm_quantized(dev(a))
    a[2, 5], a[4, 7] = np.nan, np.inf
    y = mx.rms_norm(dev(a))[0]
    q, s, _, _ = mx.rms_norm_quantized(dev(a))
    others = [0, 1, 3, 5]
    assert torch.equal(y[others], clean[others])
    assert torch.isnan(y[2]).all() and torch.isnan(q[2].float()).all()
    assert torch.equal(q[others].float(), q0[others].float()) and torch.equal(s[others], s0[others])
    # a row of zeros, with eps alone to divide by
    y, _, rstd = mx.rms_norm(torch.zeros(2, 200, device="cuda"), eps=1e-6)
    assert not y.any() and torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=1e-6)
    q, s, _, _ = mx.rms_norm_quantized(torch.zeros(2, 200, device="cuda"))
    assert not q.float().any() and (s == 1).all()


# ---------------------------------------------------------------- 8 bits
ROW_SHAPES = [(1, 1), (1, 128), (3, 7), (5, 130), (4, 512), (33, 896), (9, 1283), (2, 20000), (700, 72),
              (5000, 16)]


def _wild(shape, seed):
    """Values whose blocks differ by any factor, with zeros, subnormals and values not finite."""
    r = np.random.default_rng(seed)
    a = r.normal(size=shape) * np.exp2(r.integers(-40, 40, size=shape[:-1] + (1,)))
    flat = a.reshape(-1)
    for v in (np.nan, np.inf, -np.inf, 0.0, 1e-40, -3e38):
        flat[r.integers(0, flat.size)] = v
    if a.ndim == 2 and a.shape[0] > 2:
        a[1] = 0
        a[2] = 1e-42
    return a


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", ROW_SHAPES)
def test_quantize_rows(T, d, dtype, kind):
    say(f"quantize_rows T={T} d={d} {dtype} {kind}")
    x = dev(_wild((T, d), T * 7 + d), dtype)
    q, scales = mx.quantize_rows(x, F8[kind])
    xh = host(x)
    rs = ref.block_scales(xh, kind)
    within(scales, rs, U * rs, "scales")
    rounded(q, np.where(np.isfinite(xh), xh, np.nan) / ref.spread_rows(rs, d), 4 * U, kind, "q")
    for out in ("f32", "bf16"):
        back = mx.dequantize_rows(q, scales, DT[out])
        want = host(q) * ref.spread_rows(host(scales), d)
        fine = np.isfinite(want) & (np.abs(want) < 3.38e38)
        # the product in float32, then the storage type: below its normal numbers a rounding is
        # off by half of its smallest step (bfloat16's is 2^-133) and not relatively
        tol = (U + STORE[out]) * np.abs(want[fine]) + LEAST["f32"] + LEAST[out]
        within(host(back)[fine], want[fine], tol, "back")
        assert np.isnan(host(back)[np.isnan(want)]).all()


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,n,k", [(1, 1, 1), (2, 128, 128), (3, 129, 257), (2, 200, 64), (1, 5, 1000),
                                   (4, 136, 267), (1, 384, 8)])
def test_quantize_blocks(E, n, k, dtype, kind):
    say(f"quantize_blocks E={E} n={n} k={k} {dtype} {kind}")
    w = dev(_wild((E, n, k), E + n + k), dtype)
    q, scales = mx.quantize_blocks(w, F8[kind])
    wh = host(w)
    rs = ref.matrix_scales(wh, kind)
    assert scales.shape == rs.shape
    within(scales, rs, U * rs, "scales")
    rounded(q, np.where(np.isfinite(wh), wh, np.nan) / ref.spread_matrix(rs, n, k), 4 * U, kind, "q")


def test_every_eight_bit_value_comes_back():
    for kind, t in F8.items():
        every = torch.arange(256, dtype=torch.uint8, device="cuda").view(t)
        every = every[torch.isfinite(every.float())]
        x = torch.zeros(len(every), 128, device="cuda")
        x[:, 0], x[:, 1] = ref.F8[kind][2], every.float()       # scale 1
        q, scales = mx.quantize_rows(x, t)
        assert (scales == 1).all() and torch.equal(q[:, 1].float(), every.float()), kind
        assert torch.equal(mx.dequantize_rows(q, scales, torch.float32), x)


# ---------------------------------------------------------------- products
def _quantized(shape, seed, kind, matrices=False):
    """8-bit values of every size with scales that differ by any moderate factor."""
    r = np.random.default_rng(seed)
    q = torch.from_numpy(r.normal(size=shape).astype(np.float32) * 40).to(F8[kind])
    nb = -(-shape[-1] // 128)
    s = (shape[0], -(-shape[1] // 128), nb) if matrices else (shape[0], nb)
    scales = np.exp2(r.normal(size=s) * 3) * (1 + r.random(s))
    return q.cuda(), dev(scales)


def _product_check(M, E, n, k, offsets, dx, kind, out, label, seed=0):
    say(f"product {label} M={M} E={E} n={n} k={k} dx={dx} {kind} {out}")
    into = n if dx else k
    x, xs = _quantized((M, into), seed + 1, kind)
    w, ws = _quantized((E, n, k), seed + 2, "e4m3", True)
    call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
    oracle = ref.grouped_matmul_quantized_dx if dx else ref.grouped_matmul_quantized
    off = None if offsets is None else ints(offsets)
    y = call(x, xs, w, ws, off, DT[out])
    assert y.shape == (M, k if dx else n) and y.dtype == DT[out]
    want, size = oracle(host(x), host(xs), host(w), host(ws), [0, M] if offsets is None else offsets)
    tol = (into + into // 128 + 12) * 2 * U * size
    if out == "bf16":
        tol = tol + 2.0 ** -10 * size
        # in the mean far less: the roundings and a hundredth of them
        off_by, norm = np.linalg.norm(host(y) - want), np.linalg.norm(want)
        assert off_by <= 1.01 * STORE[out] * norm, (label, off_by / norm)
    within(y, want, tol + STORE[out] * (np.abs(want) + tol), label)
    return x, xs, w, ws, off, y


def _ragged(M, E, seed, tail=0):
    r = np.random.default_rng(seed)
    cuts = np.sort(r.integers(0, M - tail + 1, size=E - 1))
    return [0, *cuts.tolist(), M - tail]


PRODUCTS = [  # M, E, n, k
    (1, 1, 1, 1), (1, 1, 128, 128), (3, 2, 7, 5), (5, 3, 64, 128), (70, 4, 129, 130), (128, 2, 256, 384),
    (200, 3, 136, 267), (65, 1, 512, 1024), (33, 64, 96, 272), (300, 5, 320, 64), (257, 2, 272, 496),
    (700, 3, 640, 640), (1500, 2, 1040, 528), (40, 8, 1408, 2048), (1, 1, 2048, 1408), (2, 1, 30, 4111)]


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("M,E,n,k", PRODUCTS)
def test_products(M, E, n, k, dx):
    off = _ragged(M, E, M + E)
    _product_check(M, E, n, k, off, dx, "e4m3", "f32", "ragged")
    _product_check(M, E, n, k, off, dx, "e5m2", "bf16", "ragged", 10)
    if E == 1:
        _product_check(M, E, n, k, None, dx, "e4m3", "bf16", "one group", 20)


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("M,E,n,k", [(2600, 3, 1536, 1408), (4100, 60, 512, 640), (9000, 2, 768, 784)])
def test_products_of_many_tiles(M, E, n, k, dx):
    """Tile counts of several rounds, odd widths in between, e5m2 rows and float32 results."""
    _product_check(M, E, n, k, _ragged(M, E, 3, 5), dx, "e4m3", "bf16", "many tiles")
    _product_check(M, E, n, k, _ragged(M, E, 4), dx, "e5m2", "f32", "many tiles", 5)


@pytest.mark.parametrize("dx", [False, True])
def test_rows_outside_the_groups(dx):
    M, E, n, k = 150, 3, 130, 144
    offsets = [10, 60, 60, 140]
    x, xs, w, ws, off, y = _product_check(M, E, n, k, offsets, dx, "e4m3", "f32", "outside")
    assert not y[:10].any() and not y[140:].any()
    call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
    out = torch.full_like(y, 7.0)
    assert call(x, xs, w, ws, off, torch.float32, out=out) is out
    assert torch.equal(out[10:140], y[10:140]) and (out[:10] == 7).all() and (out[140:] == 7).all()
    # what stands in those rows reaches no result
    xs2 = xs.clone()
    xs2[:10], xs2[140:] = float("nan"), float("inf")
    x2 = x.clone()
    x2.view(torch.uint8)[:10] = 0x7f
    x2.view(torch.uint8)[140:] = 0x7f
    assert torch.equal(call(x2, xs2, w, ws, off, torch.float32), y)


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("offsets", [[0, 0, 0, 0], [50, 20, 70, 500], [-5, 3, 2, 90], [90, 90, 90, 90],
                                     [200, -7, 3000, 1]])
def test_offsets_that_are_empty_or_out_of_order(offsets, dx):
    _product_check(90, 3, 72, 200, offsets, dx, "e4m3", "bf16", f"offsets {offsets}")


@pytest.mark.parametrize("dx", [False, True])
def test_nan_reaches_its_own_results_only(dx):
    M, E, n, k = 40, 2, 160, 272
    x, xs, w, ws, off, y = _product_check(M, E, n, k, [0, 17, 40], dx, "e4m3", "f32", "clean")
    call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
    x.view(torch.uint8)[5, 130] = 0x7f                       # row 5
    w.view(torch.uint8)[1, 33, 144] = 0xff                   # expert 1: column 33 (dx: 144)
    z = call(x, xs, w, ws, off, torch.float32)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[5] = True
    bad[17:, 144 if dx else 33] = True
    assert torch.equal(torch.isnan(z), bad) and torch.equal(z[~bad], y[~bad])


def test_a_scale_of_any_size_belongs_to_its_block():
    M, n, k = 64, 256, 384
    x, xs = _quantized((M, k), 1, "e4m3")
    w, ws = _quantized((1, n, k), 2, "e4m3", True)
    for a, b in ((2.0 ** -100, 2.0 ** 90), (0.0, 1.0), (-1.0, 1.0), (2.0 ** 100, 2.0 ** -100)):
        xs2, ws2 = xs.clone(), ws.clone()
        xs2[:, 1] *= a
        ws2[:, :, 1] *= b
        y = mx.grouped_matmul_quantized(x, xs2, w, ws2, None, torch.float32)
        want, size = ref.grouped_matmul_quantized(host(x), host(xs2), host(w), host(ws2), [0, M])
        within(y, want, (k + 20) * 2 * U * size, f"{a} {b}")


def test_products_repeat_and_rows_do_not_depend_on_their_neighbours():
    M, E, n, k = 900, 4, 512, 640
    x, xs, w, ws, off, y = _product_check(M, E, n, k, [0, 100, 101, 600, 900], False, "e4m3", "f32", "all")
    for _ in range(3):
        assert torch.equal(mx.grouped_matmul_quantized(x, xs, w, ws, off, torch.float32), y)


def test_views_of_larger_buffers():
    """Operands that start inside a larger allocation, 16 bytes further on."""
    M, n, k = 37, 80, 133
    x, xs, w, ws, _, y = _product_check(M, 1, n, k, None, False, "e4m3", "f32", "whole")
    big = torch.zeros(M * k + 32, dtype=torch.uint8, device="cuda")
    big[16:16 + M * k] = x.view(torch.uint8).reshape(-1)
    v = big[16:16 + M * k].view(M, k).view(torch.float8_e4m3fn)
    assert torch.equal(mx.grouped_matmul_quantized(v, xs, w, ws, None, torch.float32), y)
    with pytest.raises(mx.MoEError, match="aligned"):
        mx.grouped_matmul_quantized(big[1:1 + M * k].view(M, k).view(torch.float8_e4m3fn), xs, w, ws)


# ---------------------------------------------------------------- balance loss
def _routing(T, N, K, seed):
    r = np.random.default_rng(seed)
    z = r.normal(size=(T, N)) + r.normal(size=N)
    e = np.exp(z - z.max(1, keepdims=True))
    s = (e / e.sum(1, keepdims=True)).astype(np.float32)
    return s, np.argsort(-s, 1, kind="stable")[:, :K].astype(np.int32)


def _balance_check(s, idx, offsets, mask, device_of, devices, label, seed=0):
    say(f"balance {label} T={s.shape[0]} N={s.shape[1]} K={idx.shape[1]}")
    r = np.random.default_rng(seed)
    S = 1 if offsets is None else len(offsets) - 1
    off = None if offsets is None else ints(offsets)
    m = None if mask is None else torch.tensor(mask, device="cuda")
    of = None if device_of is None else ints(device_of)
    sd, id_ = dev(s), torch.from_numpy(np.ascontiguousarray(idx)).cuda()
    a1, a2 = 0.25, 0.5
    got = mx.balance_loss(sd, id_, off, m, of, devices, a1, a2)
    want = ref.balance_loss(s, idx, offsets, mask, device_of, devices, a1, a2)
    assert np.array_equal(got["counts"].cpu().numpy(), want["counts"]), label
    # float64 sums, one rounding to float32
    for name in ("P", "losses", "slopes"):
        within(got[name], want[name], U * (1 + 1e-6) * np.abs(want[name]) + 1e-300, f"{label} {name}")
    for dl in (None, r.normal(size=(S, 2))):
        z = mx.balance_loss_backward(sd, got["slopes"], None if dl is None else dev(dl), off, m)
        sl = host(got["slopes"])
        d = np.ones((S, 2)) if dl is None else dl.astype(np.float32).astype(np.float64)
        rz = ref.balance_loss_backward(s, sl, d, offsets, mask)
        # c carries 3 u, its sum with the scores 4 + 6 additions and the products' rounding
        c = np.abs(d[:, :1] * sl[:, 0]) + np.abs(d[:, 1:] * sl[:, 1])
        tol = np.zeros_like(rz)
        for q, (a, b) in enumerate(ref.group_rows([0, s.shape[0]] if offsets is None else offsets, s.shape[0])):
            tol[a:b] = s[a:b] * (6 * U * c[q] + 20 * U * (s[a:b] @ c[q])[:, None])
        within(z, rz, tol, label + " dlogits")
        off_rows = (rz == 0).all(1) & (tol.max(1) == 0)
        assert not z[torch.from_numpy(off_rows).cuda()].any()
    return got


@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 64, 6), (7, 5, 2), (64, 63, 7), (65, 64, 6), (300, 100, 9),
                                   (1000, 128, 12), (513, 256, 16), (4096, 63, 7), (20000, 16, 3)])
def test_balance_loss(T, N, K):
    s, idx = _routing(T, N, K, T + N)
    r = np.random.default_rng(T)
    _balance_check(s, idx, None, None, None, 0, "batch")
    mask = r.random(T) < 0.7
    D = min(4, N)
    _balance_check(s, idx, None, mask, np.arange(N) * D // N, D, "masked, on devices")
    cuts = np.sort(r.integers(0, T + 1, size=5))
    _balance_check(s, idx, [0, *cuts.tolist(), T], mask, np.arange(N) % D, D, "sequences")
    _balance_check(s, idx, [T // 3, T // 2, T // 2, T - T // 4], None, None, 0, "rows of no sequence")
    _balance_check(s, idx, [0] + [min(T, 3 * i) for i in range(1, 900)] + [T], mask, np.zeros(N, int), 1,
                   "many sequences")


def test_balance_loss_of_nothing_and_of_bad_entries():
    s, idx = _routing(50, 8, 3, 1)
    _balance_check(s, idx, None, np.zeros(50, bool), np.zeros(8, int), 1, "all masked")
    _balance_check(s, idx, [0, 0, 0], None, None, 0, "empty sequences")
    _balance_check(s, idx, [60, -4, 20, 10, 99], None, None, 0, "offsets out of order")
    idx2 = idx.copy()
    idx2[3, 1], idx2[5, 0], idx2[7] = -1, 8, [2, 2, 2]          # outside; the same expert thrice
    _balance_check(s, idx2, None, None, [0, 1, 5, -1, 0, 1, 0, 1], 3, "entries outside")
    # masked rows are not read
    mask = np.ones(50, bool)
    mask[[4, 49]] = False
    clean = _balance_check(s, idx, None, mask, None, 0, "masked")
    bad = torch.from_numpy(s).cuda()
    bad[[4, 49]] = float("nan")
    got = mx.balance_loss(bad, torch.from_numpy(idx).cuda(), None, torch.from_numpy(mask).cuda(), None, 0,
                          0.25, 0.5)
    for name, v in clean.items():
        assert torch.equal(got[name], v), name
    z = mx.balance_loss_backward(bad, got["slopes"], None, None, torch.from_numpy(mask).cuda())
    assert torch.isfinite(z).all() and not z[[4, 49]].any()
    e = mx.balance_loss(torch.empty(0, 8, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    assert not any(v.any() for v in e.values())
    assert mx.balance_loss_backward(torch.empty(0, 8, device="cuda"), e["slopes"]).shape == (0, 8)


def test_balance_loss_agrees_with_the_statistics():
    s, idx = _routing(777, 63, 7, 9)
    groups = (np.arange(63) * 9 // 63).tolist()
    a = mx.balance_stats(dev(s), torch.from_numpy(idx).cuda(), 7, groups, 0.3, 0.7)
    b = mx.balance_loss(dev(s), torch.from_numpy(idx).cuda(), None, None, ints(groups), 9, 0.3, 0.7)
    assert torch.equal(a["P"], b["P"][0])
    assert torch.allclose(torch.stack([a["L_ExpBal"], a["L_DevBal"]]), b["losses"][0], rtol=2 * U)


def test_layer_backward_takes_the_balance_loss_on():
    """dlogits join dz: their part of du, dE_gate and the bias is that of the logits u E^T + b."""
    say("layer backward with dlogits")
    r = np.random.default_rng(6)
    T, d, N, K, I = 200, 128, 16, 4, 64
    for dtype in ("f32", "bf16"):
        u, E = dev(r.normal(size=(T, d)), dtype), dev(0.1 * r.normal(size=(N, d)), dtype)
        Wr = dev(0.1 * r.normal(size=N * 3 * I * d), dtype)
        dh = dev(r.normal(size=(T, d)), dtype)
        _, _, scores = mx.route(u, E, K, want_scores=True)
        idx = mx.route(u, E, K)[0]
        b = mx.balance_loss(scores, idx)
        z = mx.balance_loss_backward(scores, 50 * b["slopes"])
        plain = mx.layer_backward(u, E, Wr, None, N, K, 0, dh)
        none = mx.layer_backward(u, E, Wr, None, N, K, 0, dh, dlogits=torch.zeros_like(z))
        both = mx.layer_backward(u, E, Wr, None, N, K, 0, dh, dlogits=z)
        zh, uh, Eh = host(z), host(u), host(E)
        step = STORE[dtype]
        # the logits' gradient without z, which is rounded to the storage type for dE_gate with z
        # and without it: its roundings stand in the difference of the two results as well (ds is
        # the same in both; a tenth more for what its own roundings make of it)
        ds = np.zeros((T, N))
        for e in range(N):
            g_, c_, d_ = (host(Wr).reshape(N, 3, I * d)[e, j] for j in range(3))
            a_ = uh @ g_.reshape(I, d).T
            f = (a_ / (1 + np.exp(-a_)) * (uh @ c_.reshape(I, d).T)) @ d_.reshape(d, I).T
            ds[:, e] = np.where((idx.cpu().numpy() == e).any(1), (host(dh) * f).sum(1), 0)
        sh = host(scores)
        dz = 1.1 * np.abs(sh * (ds - (sh * ds).sum(1, keepdims=True)))
        for p_, n_, g, want, size in ((plain[0], none[0], both[0], zh @ Eh, (np.abs(zh) + 2 * dz) @ np.abs(Eh)),
                                      (plain[1], none[1], both[1], zh.T @ uh,
                                       (np.abs(zh) + 2 * dz).T @ np.abs(uh)),
                                      (plain[2], none[2], both[2], zh.sum(0), (np.abs(zh) + 2 * dz).sum(0))):
            assert torch.equal(p_, n_)
            # du is rounded once at its end; sums of at most d + N + K and T terms
            grown = 2 * host(p_).__abs__() + np.abs(want)
            tol = step * (size + 2 * grown) + 2 * (T + d) * U * (size + grown)
            within(host(g) - host(p_), want, tol, dtype)
        assert torch.equal(plain[3], both[3])                      # experts' weights do not see it


# ---------------------------------------------------------------- streams, graphs, workspaces
def _inputs_of_a_step(seed):
    x, res, w, dy, dh = _norm_inputs(70, 272, "bf16", seed)
    wq, ws = _quantized((2, 144, 272), seed + 1, "e4m3", True)
    s, idx = _routing(70, 12, 3, seed)
    return dict(x=x, res=res, w=w, dy=dy, dh=dh, wq=wq, ws=ws, off=ints([0, 30, 70]), s=dev(s),
                idx=torch.from_numpy(idx).cuda(), mask=torch.from_numpy(np.arange(70) < 64).cuda())


def _step(t):
    """Every operator once, each on what the one before it gave."""
    q, qs, h, rstd = mx.rms_norm_quantized(t["x"], t["w"], t["res"])
    y = mx.grouped_matmul_quantized(q, qs, t["wq"], t["ws"], t["off"])
    g, gs = mx.quantize_rows(y, torch.float8_e5m2)
    dq = mx.grouped_matmul_quantized_dx(g, gs, t["wq"], t["ws"], t["off"])
    dx, dw = mx.rms_norm_backward(dq, h, t["w"], rstd, t["dh"])
    wq, ws = mx.quantize_blocks(dx.view(1, 70, 272))
    b = mx.balance_loss(t["s"], t["idx"], None, t["mask"])
    z = mx.balance_loss_backward(t["s"], b["slopes"], None, None, t["mask"])
    return [q.view(torch.uint8), qs, h, rstd, y, g.view(torch.uint8), gs, dq, dx, dw, wq.view(torch.uint8),
            ws, b["counts"], b["losses"], z, mx.dequantize_rows(q, qs)]


def test_on_another_stream():
    t = _inputs_of_a_step(1)
    want = _step(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _step(t)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_and_replayed():
    """Two graphs of the same calls, with workspaces of their own, replayed in turn on new inputs
    with eager work between the replays."""
    t = _inputs_of_a_step(2)
    _step(t)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _step(t)
        graphs.append((g, out))
    for i in range(4):
        new = _inputs_of_a_step(20 + i)
        for k in t:
            if t[k].dtype in (torch.float8_e4m3fn, torch.bool):
                t[k].view(torch.uint8).copy_(new[k].view(torch.uint8))
            else:
                t[k].copy_(new[k])
        want = _step(t)
        g, out = graphs[i & 1]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_a_workspace_given_by_the_caller():
    t = _inputs_of_a_step(3)
    want = _step(t)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    ws.fill_(0xff)                                             # what lies in it does not matter
    q, qs, h, rstd = mx.rms_norm_quantized(t["x"], t["w"], t["res"])
    y = mx.grouped_matmul_quantized(q, qs, t["wq"], t["ws"], t["off"], workspace=ws)
    dq = mx.grouped_matmul_quantized_dx(*mx.quantize_rows(y, torch.float8_e5m2), t["wq"], t["ws"], t["off"],
                                        workspace=ws)
    dx, dw = mx.rms_norm_backward(dq, h, t["w"], rstd, t["dh"], workspace=ws)
    b = mx.balance_loss(t["s"], t["idx"], None, t["mask"], workspace=ws)
    for a, i in ((y, 4), (dq, 7), (dx, 8), (dw, 9), (b["losses"], 13)):
        assert torch.equal(a, want[i]), i


# ---------------------------------------------------------------- a run of them together
def test_a_training_step_of_a_block_with_experts_in_8_bits():
    """norm -> router -> 8-bit experts (SwiGLU) -> sum, with the balance loss; the gradients of the
    rows, of the experts' weights and of the norm, against float64 of the values that the 8-bit
    operands stand for (8-bit rounding passes gradients on as they are)."""
    say("a block with experts in 8 bits")
    r = np.random.default_rng(8)
    T, d, N, K, I = 150, 320, 6, 2, 144
    x, res = dev(r.normal(size=(T, d)), "bf16"), dev(r.normal(size=(T, d)), "bf16")
    wn = dev(1 + 0.1 * r.normal(size=d), "bf16")
    E = dev(0.2 * r.normal(size=(N, d)), "bf16")
    W1, W2 = dev(0.1 * r.normal(size=(N, 2 * I, d))), dev(0.1 * r.normal(size=(N, d, I)))
    (q1, s1), (q2, s2) = mx.quantize_blocks(W1), mx.quantize_blocks(W2)

    q, qs, h, rstd = mx.rms_norm_quantized(x, wn, res)
    y = mx.rms_norm(x, wn, res)[0]
    idx, gate, scores = mx.route(y, E, K, want_scores=True)
    _, off, pair = mx.dispatch(idx, N)
    tok = pair.long() // K
    xg, xgs = q.view(torch.uint8)[tok].view(q.dtype), qs[tok]
    a = mx.grouped_matmul_quantized(xg, xgs, q1, s1, off, torch.float32)
    p_ = torch.nn.functional.silu(a[:, :I]) * a[:, I:] * gate.reshape(-1)[pair.long()][:, None]
    pq, ps = mx.quantize_rows(p_)
    o = mx.grouped_matmul_quantized(pq, ps, q2, s2, off)
    Y = torch.empty_like(o)
    Y[pair.long()] = o
    out = mx.combine(h, Y, None, K, 0)
    # float64 of the same operands
    rows = off.cpu().numpy()
    a64, size = ref.grouped_matmul_quantized(host(xg), host(xgs), host(q1), host(s1), rows)
    within(a, a64, (d + 20) * 2 * U * size + U * np.abs(a64), "gate and up")
    o64, osize = ref.grouped_matmul_quantized(host(pq), host(ps), host(q2), host(s2), rows)
    place = np.argsort(pair.cpu().numpy())
    oerr = 2.0 ** -8 * np.abs(o64) + (2.0 ** -10 + (I + 20) * 2 * U) * osize
    h64 = host(h) + o64[place].reshape(T, K, d).sum(1)
    within(out, h64, 2.0 ** -8 * np.abs(h64) + 1.01 * oerr[place].reshape(T, K, d).sum(1) + 1e-6, "out")

    # backward of o's and a's products and of the norm
    dout = dev(r.normal(size=(T, d)), "bf16")
    do = dout[tok].contiguous()
    dpq, dps = mx.quantize_rows(do, torch.float8_e5m2)
    dp = mx.grouped_matmul_quantized_dx(dpq, dps, q2, s2, off, torch.float32)
    dp64, size = ref.grouped_matmul_quantized_dx(host(dpq), host(dps), host(q2), host(s2), rows)
    within(dp, dp64, (d + 20) * 2 * U * size + U * np.abs(dp64), "dp")
    # the weights' gradient from the rows that were kept in 8 bits
    pb = mx.dequantize_rows(pq, ps)
    _, dW2 = mx.grouped_matmul_backward(pb, W2.bfloat16(), off, do, need_dx=False)
    _, dw64 = ref.grouped_matmul_backward(host(pb), host(W2), rows, host(do))
    _, dwsize = ref.grouped_matmul_backward(abs(host(pb)), host(W2), rows, abs(host(do)))
    within(dW2, dw64, (T * K + 8) * 2 * U * dwsize, "dW2")
    da = dev(r.normal(size=(T * K, 2 * I)), "bf16")
    daq, das = mx.quantize_rows(da, torch.float8_e5m2)
    dxg = mx.grouped_matmul_quantized_dx(daq, das, q1, s1, off, torch.float32)
    dy = torch.zeros(T, d, device="cuda").index_add_(0, tok, dxg).bfloat16()
    dx, dwn = mx.rms_norm_backward(dy, h, wn, rstd, dout)
    _norm_backward_check(dy, h, wn, rstd, dout, "bf16", "norm")
    b = mx.balance_loss(scores, idx)
    z = mx.balance_loss_backward(scores, b["slopes"])
    # a softmax's gradient sums to nothing in each row: N + 6 roundings of s (|c| + |s c|)
    assert (z.double().sum(1).abs() <= 40 * U * b["slopes"][0, 0].abs().max()).all()
