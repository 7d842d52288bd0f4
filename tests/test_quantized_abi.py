"""Refusals of the operators for 8-bit experts and of the balance loss, on the CPU: bad arguments
are rejected before anything touches the GPU (every call below ends in a validation error or is
empty)."""
import ctypes
import os

import pytest
import torch

mx = pytest.importorskip("mixture_experts_ffn_fp32_amd")
from mixture_experts_ffn_fp32_amd import moe as binding  # noqa: E402

OK, INVALID, UNSUPPORTED, WORKSPACE, ALIGNMENT = 0, 1, 2, 3, 4
F32, BF16, E4M3, E5M2 = 0, 1, 2, 3
BIG = 1 << 44
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.fail("libmoe.so is not built: run python -m mixture_experts_ffn_fp32_amd.build")
    return binding.load_library()


def p(x):
    return None if x is None else ctypes.c_void_p(x)


def size(query, *args):
    out = ctypes.c_size_t(0)
    status = query(*args, ctypes.byref(out))
    return status, out.value


def says(lib, text):
    return text in lib.moe_last_error().decode()


# ---------------------------------------------------------------- RMS norm
def _rms(lib, x=1 << 20, res=1 << 21, w=16, T=4, d=64, eps=1e-6, dt=BF16, yt=BF16, h=1 << 22,
         y=1 << 24, scales=None, rstd=1 << 27):
    return lib.moe_rms_norm(p(x), p(res), p(w), T, d, eps, dt, yt, p(h), p(y), p(scales), p(rstd), None)


def test_rms_norm_refusals(lib):
    assert _rms(lib, T=-1) == INVALID
    assert _rms(lib, d=0) == INVALID
    assert _rms(lib, d=(1 << 24) + 1) == UNSUPPORTED
    assert _rms(lib, dt=E4M3) == UNSUPPORTED and _rms(lib, yt=F32) == UNSUPPORTED
    assert _rms(lib, yt=4) == UNSUPPORTED
    for eps in (-1e-6, NAN, INF):
        assert _rms(lib, eps=eps) == INVALID
    assert _rms(lib, x=None) == INVALID and says(lib, "x is NULL")
    assert _rms(lib, y=None) == INVALID
    assert _rms(lib, scales=1 << 28) == INVALID and says(lib, "8-bit")
    assert _rms(lib, yt=E4M3) == INVALID and says(lib, "scales is NULL")
    for name in ("x", "res", "w", "h", "y", "rstd"):
        assert _rms(lib, **{name: (1 << 30) + 8}) == ALIGNMENT, name
    assert _rms(lib, yt=E5M2, scales=(1 << 30) + 4) == ALIGNMENT
    assert _rms(lib, y=1 << 20) == INVALID and says(lib, "y overlaps x")
    assert _rms(lib, y=1 << 21) == INVALID and says(lib, "y overlaps residual")
    assert _rms(lib, h=(1 << 20) + 16) == INVALID and says(lib, "h overlaps x")
    assert _rms(lib, h=(1 << 21) + 4 * 64 * 2 - 16) == INVALID
    assert _rms(lib, h=1 << 20, y=1 << 20) == INVALID             # h in x's place, y as well
    assert _rms(lib, rstd=1 << 24) == INVALID
    assert _rms(lib, yt=E4M3, scales=1 << 24) == INVALID and says(lib, "overlaps")
    assert _rms(lib, T=0, x=None, y=None) == OK


def _rms_bwd(lib, dy=1 << 20, h=1 << 21, w=16, rstd=1 << 22, dh=1 << 23, T=4, d=64, dt=BF16,
             dx=1 << 24, dw=1 << 25, ws=BIG, wsb=1 << 40):
    return lib.moe_rms_norm_backward(p(dy), p(h), p(w), p(rstd), p(dh), T, d, dt, p(dx), p(dw), p(ws),
                                     wsb, None)


def test_rms_norm_backward_refusals(lib):
    query = lib.moe_rms_norm_backward_workspace_size
    status, need = size(query, 4, 64, BF16)
    assert status == OK and need > 0
    assert size(query, 0, 64, BF16) == (OK, 0)
    # rows too long for registers: partial rows of T / 1024 rows each, up to the largest T
    assert size(query, 2 ** 31 - 1, 20000, F32) == (OK, 1024 * 20000 * 4)
    assert size(query, 4, 0, BF16)[0] == INVALID
    assert query(4, 64, BF16, None) == INVALID
    for name in ("dy", "h", "rstd", "dx", "ws"):
        assert _rms_bwd(lib, **{name: None}) == INVALID, name
    for name in ("dy", "h", "w", "rstd", "dh", "dx", "dw", "ws"):
        assert _rms_bwd(lib, **{name: (1 << 30) + 4}) == ALIGNMENT, name
    assert _rms_bwd(lib, wsb=need - 1) == WORKSPACE
    assert _rms_bwd(lib, dx=1 << 20) == INVALID and says(lib, "dx overlaps dy")
    assert _rms_bwd(lib, dx=1 << 21) == INVALID and says(lib, "dx overlaps h")
    assert _rms_bwd(lib, dx=(1 << 23) + 16) == INVALID and says(lib, "dx overlaps dh")
    assert _rms_bwd(lib, dw=BIG) == INVALID
    assert _rms_bwd(lib, dt=E5M2) == UNSUPPORTED
    # an empty batch without a weight gradient has nothing to do
    assert _rms_bwd(lib, T=0, dy=None, h=None, rstd=None, dh=None, dx=None, dw=None, ws=None,
                    wsb=0) == OK


# ---------------------------------------------------------------- 8 bits
def test_quantize_refusals(lib):
    def rows(x=1 << 20, T=4, d=64, dt=BF16, qt=E4M3, q=1 << 22, s=1 << 23):
        return lib.moe_quantize_rows(p(x), T, d, dt, qt, p(q), p(s), None)

    def blocks(w=1 << 24, E=2, n=64, k=64, dt=F32, qt=E4M3, q=1 << 26, s=1 << 27):
        return lib.moe_quantize_blocks(p(w), E, n, k, dt, qt, p(q), p(s), None)

    def back(q=1 << 20, s=1 << 21, T=4, d=64, qt=E4M3, dt=BF16, x=1 << 22):
        return lib.moe_dequantize_rows(p(q), p(s), T, d, qt, dt, p(x), None)

    for call in (rows, back):
        assert call(T=-1) == INVALID and call(d=0) == INVALID
        assert call(d=(1 << 24) + 1) == UNSUPPORTED
    for call in (rows, blocks, back):
        assert call(qt=BF16) == UNSUPPORTED and call(dt=E4M3) == UNSUPPORTED
        for name in ("q", "s"):
            assert call(**{name: None}) == INVALID, name
            assert call(**{name: (1 << 30) + 8}) == ALIGNMENT, name
    assert rows(x=None) == INVALID and blocks(w=None) == INVALID and back(x=None) == INVALID
    assert rows(q=1 << 20) == INVALID and says(lib, "q overlaps x")
    assert rows(s=1 << 22) == INVALID
    assert blocks(q=(1 << 24) + 16) == INVALID and blocks(s=1 << 26) == INVALID
    assert back(x=1 << 20) == INVALID and back(x=1 << 21) == INVALID
    assert blocks(E=-1) == INVALID and blocks(n=0) == INVALID and blocks(k=0) == INVALID
    assert blocks(n=(1 << 20) + 1) == UNSUPPORTED
    assert blocks(E=129, n=1 << 15, k=1 << 15) == UNSUPPORTED and says(lib, "2^23 blocks")
    assert rows(T=0, x=None) == OK and back(T=0, x=None) == OK and blocks(E=0, w=None) == OK


def test_quantized_product_refusals(lib):
    def y(x=1 << 30, xs=1 << 31, w=1 << 32, ws=1 << 33, off=16, M=64, E=4, n=128, k=64, xt=E4M3,
          ot=BF16, out=1 << 34, wsp=BIG, wsb=1 << 40):
        return lib.moe_grouped_matmul_quantized(p(x), p(xs), p(w), p(ws), p(off), M, E, n, k, xt, ot,
                                                1, p(out), p(wsp), wsb, None)

    def dx(x=1 << 30, xs=1 << 31, w=1 << 32, ws=1 << 33, off=16, M=64, E=4, n=128, k=64, xt=E4M3,
           ot=BF16, out=1 << 34, wsp=BIG, wsb=1 << 40):
        return lib.moe_grouped_matmul_quantized_dx(p(x), p(xs), p(w), p(ws), p(off), M, E, n, k, xt,
                                                   ot, 1, p(out), p(wsp), wsb, None)

    shapes = [((-1, 4, 8, 8), INVALID), ((8, 0, 8, 8), INVALID), ((8, 4, 0, 8), INVALID),
              ((8, 4, 8, 0), INVALID), ((8, 1025, 8, 8), UNSUPPORTED),
              ((8, 4, (1 << 20) + 1, 8), UNSUPPORTED), ((8, 4, 8, (1 << 20) + 1), UNSUPPORTED),
              ((2 ** 31 - 1, 1024, 1 << 20, 1 << 20), UNSUPPORTED)]
    for call, query in ((y, lib.moe_grouped_matmul_quantized_workspace_size),
                        (dx, lib.moe_grouped_matmul_quantized_dx_workspace_size)):
        for (M, E, n, k), want in shapes:
            assert size(query, M, E, n, k)[0] == want, (M, E, n, k)
            assert call(M=M, E=E, n=n, k=k) == want
        assert query(8, 4, 8, 8, None) == INVALID
        assert size(query, 0, 4, 8, 8) == (OK, 0)
        assert call(xt=BF16) == UNSUPPORTED and call(ot=E4M3) == UNSUPPORTED
        for name in ("x", "xs", "w", "ws", "off", "out"):
            assert call(**{name: None}) == INVALID, name
            assert call(**{name: (1 << 38) + 8}) == ALIGNMENT, name
        for name, at in (("x", 1 << 30), ("xs", 1 << 31), ("w", 1 << 32), ("ws", 1 << 33)):
            assert call(out=at) == INVALID and says(lib, "overlaps"), name
        assert call(E=1, off=None, M=0) == OK
        assert call(M=0, x=None, xs=None, out=None) == OK
        # odd rows: copied, or where they are few (and hold 16 bytes) read in place
        assert size(query, 64, 4, 136, 267) == (OK, 0) and size(query, 1, 1, 2041, 1407) == (OK, 0)
        assert size(query, 64, 4, 13, 7)[1] > 0 and size(query, 20000, 4, 136, 267)[1] > 0
        status, need = size(query, 64, 4, 13, 7)
        assert status == OK
        assert call(M=64, n=13, k=7, wsb=need - 1) == WORKSPACE
        assert call(M=64, n=13, k=7, wsp=None) == INVALID
        assert call(M=64, n=13, k=7, wsp=1 << 34) == INVALID and says(lib, "overlaps")


# ---------------------------------------------------------------- balance loss
def test_balance_loss_refusals(lib):
    query = lib.moe_balance_loss_workspace_size

    def fwd(sc=1 << 20, idx=1 << 22, off=16, mask=1 << 12, dev=1 << 13, T=64, N=8, K=2, S=3, D=2,
            a1=1.0, a2=1.0, cnt=1 << 24, P=1 << 25, loss=1 << 26, sl=1 << 27, ws=BIG, wsb=1 << 40):
        return lib.moe_balance_loss(p(sc), p(idx), p(off), p(mask), p(dev), T, N, K, S, D, a1, a2,
                                    p(cnt), p(P), p(loss), p(sl), p(ws), wsb, None)

    def bwd(sc=1 << 20, sl=1 << 22, dl=1 << 23, off=16, mask=1 << 12, T=64, N=8, S=3, z=1 << 24):
        return lib.moe_balance_loss_backward(p(sc), p(sl), p(dl), p(off), p(mask), T, N, S, p(z), None)

    status, need = size(query, 64, 8, 3)
    assert status == OK and need > 0
    assert size(query, 0, 8, 3) == (OK, 0)
    assert query(64, 8, 3, None) == INVALID
    for call in (fwd, bwd):
        assert call(T=-1) == INVALID and call(N=0) == INVALID and call(S=0) == INVALID
        assert call(N=257) == UNSUPPORTED and call(S=1025) == UNSUPPORTED
        assert call(off=None) == INVALID                     # three sequences need their offsets
        for name in ("sc", "off", "mask", "sl"):
            assert call(**{name: (1 << 30) + 8}) == ALIGNMENT, name
        for name in ("sc", "sl"):
            assert call(**{name: None}) == INVALID, name
    assert fwd(K=0) == INVALID and fwd(K=9) == INVALID
    assert fwd(D=-1) == INVALID and fwd(D=257) == UNSUPPORTED
    assert fwd(D=0) == INVALID and says(lib, "device_of needs")
    assert fwd(T=2 ** 30, K=2) == UNSUPPORTED
    for a in (NAN, INF):
        assert fwd(a1=a) == INVALID and fwd(a2=a) == INVALID
    for name in ("idx", "cnt", "P", "loss", "ws"):
        assert fwd(**{name: None}) == INVALID, name
        assert fwd(**{name: (1 << 30) + 8}) == ALIGNMENT, name
    assert fwd(wsb=need - 1) == WORKSPACE
    assert fwd(P=1 << 24) == INVALID and says(lib, "overlaps")
    assert fwd(cnt=1 << 20) == INVALID and fwd(sl=BIG) == INVALID
    assert bwd(z=None) == INVALID and bwd(z=1 << 20) == INVALID and bwd(z=1 << 22) == INVALID
    assert bwd(T=0, sc=None, z=None) == OK


def test_layer_backward_with_logit_gradients_refusals(lib):
    def bwd(z, du=1 << 33, ws=BIG):
        return lib.moe_layer_backward_aux(p(1 << 30), p(1 << 31), p(1 << 32), None, 4, 2, 0, 8, 64,
                                          64, BF16, None, p((1 << 32) + (1 << 31)), p(z), p(du),
                                          p(1 << 34), None, p(1 << 35), None, p(ws), 1 << 40, None)

    assert bwd((1 << 36) + 4) == ALIGNMENT
    for at in (1 << 33, 1 << 34, 1 << 35, BIG):
        assert bwd(at) == INVALID and says(lib, "dlogits overlaps")


# ---------------------------------------------------------------- the binding
def test_the_binding_refuses_before_the_library_is_called():
    x, q = torch.zeros(4, 130), torch.zeros(4, 130).to(torch.float8_e4m3fn)
    w = torch.zeros(2, 6, 130).to(torch.float8_e4m3fn)
    xs, ws, off = torch.ones(4, 2), torch.ones(2, 1, 2), torch.zeros(3, dtype=torch.int32)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    cases = [
        (lambda: mx.rms_norm(x), "GPU"),
        (lambda: mx.rms_norm(x, residual=x[:2]), "shape"),
        (lambda: mx.rms_norm(x, weight=x[0].double()), "dtype"),
        (lambda: mx.rms_norm(x.half()), "unsupported"),
        (lambda: mx.rms_norm_quantized(x, q_dtype=torch.int8), "float8"),
        (lambda: mx.rms_norm_backward(x, x, None, torch.ones(3)), "shape"),
        (lambda: mx.rms_norm_backward(x, x, None, torch.ones(4), dh=x[0]), "shape"),
        (lambda: mx.quantize_rows(x[0]), "dimensions"),
        (lambda: mx.quantize_rows(x), "GPU"),
        (lambda: mx.quantize_blocks(x), "dimensions"),
        (lambda: mx.dequantize_rows(x, xs), "float8"),
        (lambda: mx.dequantize_rows(q, xs[:, :1]), "shape"),
        (lambda: mx.dequantize_rows(q, xs, torch.float16), "unsupported"),
        (lambda: mx.grouped_matmul_quantized(q, xs, w, ws, off), "GPU"),
        (lambda: mx.grouped_matmul_quantized(q[:, :128], xs, w, ws, off), "rows of 128"),
        (lambda: mx.grouped_matmul_quantized(x, xs, w, ws, off), "float8"),
        (lambda: mx.grouped_matmul_quantized(q, xs, w.view(torch.float8_e5m2), ws, off), "e4m3"),
        (lambda: mx.grouped_matmul_quantized(q, xs[:, :1], w, ws, off), "shape"),
        (lambda: mx.grouped_matmul_quantized(q, xs, w, ws[:1], off), "shape"),
        (lambda: mx.grouped_matmul_quantized(q, xs, w, ws, None), "offsets"),
        (lambda: mx.grouped_matmul_quantized(q, xs, w, ws, off.long()), "dtype"),
        (lambda: mx.grouped_matmul_quantized(q, xs, w, ws, off, torch.float16), "unsupported"),
        (lambda: mx.grouped_matmul_quantized_dx(q, xs, w, ws, off), "rows of 130"),
        (lambda: mx.balance_loss(x, idx), "GPU"),
        (lambda: mx.balance_loss(x, idx.long()), "dtype"),
        (lambda: mx.balance_loss(x, idx[:2]), "shape"),
        (lambda: mx.balance_loss(x, idx, mask=torch.ones(4)), "dtype"),
        (lambda: mx.balance_loss_backward(x, torch.ones(1, 130)), "shape"),
        (lambda: mx.balance_loss_backward(x, torch.ones(2, 2, 130), offsets=off, dlosses=x), "shape"),
    ]
    for call, text in cases:
        with pytest.raises(mx.MoEError) as e:
            call()
        assert text in e.value.message, (text, e.value.message)
