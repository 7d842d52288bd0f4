"""8-bit products whose two scales multiply to more than float32 holds: each result is finite,
infinite or NaN as its own value is.  Tolerances as in test_gpu_quantized.py."""
import numpy as np
import pytest
import torch

from oracle import operators as ref
from parity_helpers import say
from test_gpu_quantized import DT, F8, STORE, U, _quantized, _ragged, dev, host, ints

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mixture_experts_ffn_fp32_amd")

# M, E, n, k: tiles of 64^2, odd rows in place, 64^2, copied odd rows in 128^2, 128^2, 256^2 and y of 256^2
# with a cut last round (bfloat16 results)
SHAPES = [(40, 2, 144, 272), (70, 1, 130, 261), (700, 3, 1040, 1040), (5000, 2, 1030, 1037), (5000, 3, 2064, 2064), (6000, 3, 2064, 2064),
          (5200, 4, 4208, 272)]
TOP = {"f32": float(np.finfo(np.float32).max), "bf16": float(torch.finfo(torch.bfloat16).max)}


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("M,E,n,k", SHAPES)
def test_scales_whose_product_leaves_float32(M, E, n, k, dx, out):
    say(f"far scales M={M} E={E} n={n} k={k} dx={dx} {out}")
    kind = "e5m2" if dx else "e4m3"
    into, width = (n, k) if dx else (k, n)
    offsets = _ragged(M, E, M, 2)
    x, xs = _quantized((M, into), 1, kind)
    w, ws = _quantized((E, n, k), 2, "e4m3", True)
    # one block of w along the contraction, for every second block of columns, is large
    big = ws[:, 1, ::2] if dx else ws[:, ::2, 1]
    big.fill_(2.0 ** 76 / 448)
    call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
    oracle = ref.grouped_matmul_quantized_dx if dx else ref.grouped_matmul_quantized
    off = ints(offsets)
    plain = call(x, xs, w, ws, off, DT[out])
    # every seventh row has a large scale there, beside zeros, one small value, or anything
    rows = np.arange(3, M, 7)
    zero, small, large = rows[0::3], rows[1::3], rows[2::3]
    xv = x.float()
    part = slice(128, min(256, into))
    xv[zero, part] = 0                              # 0 times infinity, were the scales multiplied
    xv[small, part] = 0
    xv[small, 128] = 2.0 ** -9                      # finite: at most 2^-9 2^8 2^146 / 448^2 = 2^127.4
    xs[rows, 1] = 2.0 ** 70 / 448
    x = xv.to(F8[kind])
    y = call(x, xs, w, ws, off, DT[out])
    want, size = oracle(host(x), host(xs), host(w), host(ws), offsets)
    tol = (into + into // 128 + 12) * 2 * U * size + (2.0 ** -10 * size if out == "bf16" else 0)
    got, want = host(y), np.asarray(want)
    inside = np.abs(want) + tol < TOP[out]
    outside = np.abs(want) - tol > TOP[out] * (1 + 2.0 ** -8)
    assert inside[zero].all() and inside[small].all() and outside[large].any()
    assert not np.isnan(got).any()
    err = np.abs(np.where(inside, got, 0) - np.where(inside, want, 0))
    assert (err <= np.where(inside, tol + STORE[out] * (np.abs(want) + tol), 0)).all()
    assert np.isfinite(got[inside]).all()
    assert (got[outside] == np.sign(want[outside]) * np.inf).all()
    # the other rows have the bits that they have without these
    rest = np.setdiff1d(np.arange(M), rows)
    assert torch.equal(y[rest], plain[rest])


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("M,E,n,k", SHAPES)
def test_far_scales_beside_values_that_are_not_finite(M, E, n, k, dx):
    """NaN and infinite scales and NaN values stay what they are, in their own results."""
    say(f"far scales and NaN M={M} E={E} n={n} k={k} dx={dx}")
    into, width = (n, k) if dx else (k, n)
    x, xs = _quantized((M, into), 1, "e4m3")
    w, ws = _quantized((E, n, k), 2, "e4m3", True)
    off = ints(_ragged(M, E, M))
    call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
    y = call(x, xs, w, ws, off)
    x.view(torch.uint8)[5, 128] = 0x7f              # NaN
    xs[6, 1] = float("nan")
    xs[7, 1] = float("inf")                         # inf times a sum: +-inf, and NaN for a sum of 0
    xs[8, 1] = 2.0 ** 126
    z = call(x, xs, w, ws, off)
    assert torch.isnan(z[5]).all() and torch.isnan(z[6]).all() and not torch.isfinite(z[7]).any()
    rest = [i for i in range(M) if not 5 <= i <= 8]
    assert torch.equal(z[rest], y[rest])
    ws.fill_(2.0 ** 80)                             # every scale's product with row 8's leaves the range
    z = call(x, xs, w, ws, off)
    assert torch.isnan(z[5]).all() and torch.isnan(z[6]).all() and not torch.isfinite(z[7]).any()
    xz = x.clone()
    xz.view(torch.uint8)[8, 128:min(256, into)] = 0
    z = call(xz, xs, w, ws, off)
    assert torch.isfinite(z[8]).all()
