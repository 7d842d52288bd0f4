"""Refusals of the operators beside the layer, on the CPU: bad arguments are rejected before
anything touches the GPU (every call below ends in a validation error or is empty)."""
import ctypes
import itertools
import os

import pytest
import torch

mx = pytest.importorskip("mixture_experts_ffn_fp32_amd")
from mixture_experts_ffn_fp32_amd import moe as binding  # noqa: E402

OK, INVALID, UNSUPPORTED, WORKSPACE, ALIGNMENT = 0, 1, 2, 3, 4
BIG = 1 << 44


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


# ---------------------------------------------------------------- layer norm
def _norm(lib, x=1 << 20, w=16, b=1 << 12, T=4, d=64, eps=1e-5, dt=1, y=1 << 24, mean=1 << 26,
          rstd=1 << 27):
    return lib.moe_layer_norm(p(x), p(w), p(b), T, d, eps, dt, p(y), p(mean), p(rstd), None)


def test_layer_norm_refusals(lib):
    assert _norm(lib, T=-1) == INVALID
    assert _norm(lib, d=0) == INVALID
    assert _norm(lib, d=(1 << 24) + 1) == UNSUPPORTED
    assert _norm(lib, dt=2) == UNSUPPORTED
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _norm(lib, eps=eps) == INVALID
    assert _norm(lib, x=None) == INVALID and says(lib, "x is NULL")
    assert _norm(lib, y=None) == INVALID
    for name in ("x", "w", "b", "y", "mean", "rstd"):
        assert _norm(lib, **{name: (1 << 30) + 8}) == ALIGNMENT, name
    assert _norm(lib, y=1 << 20) == INVALID and says(lib, "y overlaps x")
    assert _norm(lib, y=(1 << 20) + 4 * 64 * 2 - 16) == INVALID          # its last 16 bytes
    assert _norm(lib, mean=1 << 24) == INVALID
    assert _norm(lib, rstd=1 << 26) == INVALID
    assert _norm(lib, T=0, x=None, y=None) == OK


def _norm_bwd(lib, dy=1 << 20, x=1 << 21, w=16, mean=1 << 22, rstd=1 << 23, T=4, d=64, dt=1,
              dx=1 << 24, dw=1 << 25, db=1 << 26, ws=BIG, wsb=1 << 40):
    return lib.moe_layer_norm_backward(p(dy), p(x), p(w), p(mean), p(rstd), T, d, dt, p(dx), p(dw),
                                       p(db), p(ws), wsb, None)


def test_layer_norm_backward_refusals(lib):
    query = lib.moe_layer_norm_backward_workspace_size
    status, need = size(query, 4, 64, 1)
    assert status == OK and need > 0
    assert size(query, 0, 64, 1) == (OK, 0)
    assert size(query, 4, 0, 1)[0] == INVALID
    assert query(4, 64, 1, None) == INVALID
    for name in ("dy", "x", "mean", "rstd", "dx", "ws"):
        assert _norm_bwd(lib, **{name: None}) == INVALID, name
    for name in ("dy", "x", "w", "mean", "rstd", "dx", "dw", "db", "ws"):
        assert _norm_bwd(lib, **{name: (1 << 30) + 4}) == ALIGNMENT, name
    assert _norm_bwd(lib, wsb=need - 1) == WORKSPACE
    assert _norm_bwd(lib, dx=1 << 20) == INVALID and says(lib, "dx overlaps dy")
    assert _norm_bwd(lib, dw=1 << 26) == INVALID
    assert _norm_bwd(lib, dw=BIG) == INVALID and says(lib, "overlaps")
    assert _norm_bwd(lib, dt=7) == UNSUPPORTED
    # an empty batch without weight gradients has nothing to do
    assert _norm_bwd(lib, T=0, dy=None, x=None, mean=None, rstd=None, dx=None, dw=None, db=None,
                     ws=None, wsb=0) == OK


# ---------------------------------------------------------------- grouped products
def _grouped(lib, x=1 << 30, w=1 << 32, off=16, M=64, E=4, n=128, k=64, dt=1, rest=1, y=1 << 34,
             ws=BIG, wsb=1 << 40):
    return lib.moe_grouped_matmul(p(x), p(w), p(off), M, E, n, k, dt, rest, p(y), p(ws), wsb, None)


def _grouped_bwd(lib, x=1 << 30, w=1 << 32, off=16, dy=1 << 33, M=64, E=4, n=128, k=64, dt=0,
                 dx=1 << 34, dw=1 << 35, ws=BIG, wsb=1 << 40):
    return lib.moe_grouped_matmul_backward(p(x), p(w), p(off), p(dy), M, E, n, k, dt, 1, p(dx), p(dw),
                                           p(ws), wsb, None)


def test_grouped_refusals(lib):
    shapes = [((-1, 4, 8, 8, 0), INVALID), ((8, 0, 8, 8, 0), INVALID), ((8, 4, 0, 8, 0), INVALID),
              ((8, 4, 8, 0, 0), INVALID), ((8, 1025, 8, 8, 0), UNSUPPORTED),
              ((8, 4, (1 << 20) + 1, 8, 0), UNSUPPORTED), ((8, 4, 8, (1 << 20) + 1, 1), UNSUPPORTED),
              ((8, 4, 8, 8, 2), UNSUPPORTED), ((2 ** 31 - 1, 1024, 1 << 20, 1 << 20, 1), UNSUPPORTED)]
    for (M, E, n, k, dt), want in shapes:
        assert size(lib.moe_grouped_matmul_workspace_size, M, E, n, k, dt)[0] == want, (M, E, n, k)
        assert size(lib.moe_grouped_matmul_backward_workspace_size, M, E, n, k, dt, 1, 1)[0] == want
        assert _grouped(lib, M=M, E=E, n=n, k=k, dt=dt) == want
        assert _grouped_bwd(lib, M=M, E=E, n=n, k=k, dt=dt) == want
    assert lib.moe_grouped_matmul_workspace_size(8, 4, 8, 8, 0, None) == INVALID
    assert lib.moe_grouped_matmul_backward_workspace_size(8, 4, 8, 8, 0, 1, 1, None) == INVALID
    for name in ("x", "w", "off", "y"):
        assert _grouped(lib, **{name: None}) == INVALID, name
        assert _grouped(lib, **{name: (1 << 38) + 8}) == ALIGNMENT, name
    assert _grouped(lib, y=1 << 30) == INVALID and says(lib, "y overlaps x")
    assert _grouped(lib, y=(1 << 32) + 64) == INVALID and says(lib, "y overlaps w")
    assert _grouped(lib, dt=0, ws=1 << 34) == INVALID                     # the workspace overlaps y
    need = size(lib.moe_grouped_matmul_workspace_size, 64, 4, 128, 64, 0)[1]
    assert need > 0
    assert _grouped(lib, dt=0, wsb=need - 1) == WORKSPACE
    assert _grouped(lib, dt=0, ws=None) == INVALID
    assert _grouped(lib, M=0, x=None, y=None, ws=None, wsb=0) == OK


def test_grouped_backward_refusals(lib):
    assert _grouped_bwd(lib, dx=None, dw=None) == INVALID and says(lib, "nothing to compute")
    for name in ("off", "dy", "x", "w"):
        assert _grouped_bwd(lib, **{name: None}) == INVALID, name
    for name in ("x", "w", "off", "dy", "dx", "dw", "ws"):
        assert _grouped_bwd(lib, **{name: (1 << 38) + 4}) == ALIGNMENT, name
    assert _grouped_bwd(lib, dx=1 << 33) == INVALID and says(lib, "dx overlaps dy")
    assert _grouped_bwd(lib, dw=1 << 34) == INVALID
    assert _grouped_bwd(lib, ws=1 << 35) == INVALID
    need = size(lib.moe_grouped_matmul_backward_workspace_size, 64, 4, 128, 64, 0, 1, 1)[1]
    assert _grouped_bwd(lib, wsb=need - 1) == WORKSPACE
    # one gradient needs its own operands only
    assert _grouped_bwd(lib, x=None, dw=None, wsb=0) == WORKSPACE
    assert _grouped_bwd(lib, w=None, dx=None, wsb=0) == WORKSPACE
    assert _grouped_bwd(lib, M=0, dw=None, x=None, w=None, dy=None, off=None, ws=None, wsb=0) == OK


def test_grouped_backward_of_an_empty_batch_needs_no_dx_pointer(lib):
    """dx of no rows has no elements, and a framework's empty tensor no address."""
    for dt in (0, 1):
        assert _grouped_bwd(lib, M=0, dt=dt, dx=None, dw=None, x=None, w=None, dy=None, ws=None, wsb=0) == OK
        assert _grouped_bwd(lib, M=1, dt=dt, dx=None, dw=None) == INVALID


def test_workspaces_grow_with_the_rows(lib):
    """A workspace for the largest batch holds every smaller one."""
    rows = [0, 1, 2, 31, 64, 65, 127, 500, 512, 513, 4096, 8191, 8192, 100_000]
    for dt, d in itertools.product((0, 1), (1, 64, 1283, 5000, 20000)):
        got = [size(lib.moe_layer_norm_backward_workspace_size, T, d, dt) for T in rows]
        assert all(s == OK for s, _ in got) and [b for _, b in got] == sorted(b for _, b in got), d
    for dt, (E, n, k) in itertools.product((0, 1), ((1, 8, 8), (64, 1408, 2048), (7, 33, 100))):
        for args in ((), (1, 0), (0, 1), (1, 1)):
            query = (lib.moe_grouped_matmul_backward_workspace_size if args
                     else lib.moe_grouped_matmul_workspace_size)
            got = [size(query, M, E, n, k, dt, *args) for M in rows]
            assert all(s == OK for s, _ in got), (E, n, k, args)
            assert [b for _, b in got] == sorted(b for _, b in got), (E, n, k, dt, args)


def test_float32_workspaces_grow_across_the_few_rows_rules(lib):
    for n, k in itertools.product((32, 33, 36, 64, 68, 100, 1408), (4, 96, 192, 252, 256, 260, 2048)):
        for E in (1, 3, 64):
            rows = sorted({r * E + d for r in (1, 63, 64, 65, 127, 128, 129, 300) for d in (-1, 0, 1)})
            for args in ((), (1, 0), (0, 1), (1, 1)):
                query = (lib.moe_grouped_matmul_backward_workspace_size if args
                         else lib.moe_grouped_matmul_workspace_size)
                got = [size(query, M, E, n, k, 0, *args)[1] for M in rows]
                assert got == sorted(got), (E, n, k, args, got)


# ---------------------------------------------------------------- orthogonalised update
def _ortho(lib, x=1 << 30, xs=64 * 128, B=2, m=64, n=128, dt=0, steps=5, eps=1e-7, a=3.4445,
           b=-4.7750, c=2.0315, out=1 << 34, os_=64 * 128, odt=0, ws=BIG, wsb=1 << 40):
    return lib.moe_orthogonalize(p(x), xs, B, m, n, dt, steps, eps, a, b, c, p(out), os_, odt, p(ws),
                                 wsb, None)


def test_orthogonalize_refusals(lib):
    query = lib.moe_orthogonalize_workspace_size
    for (B, m, n), want in [((-1, 8, 8), INVALID), ((1, 0, 8), INVALID), ((1, 8, 0), INVALID),
                            ((65536, 8, 8), UNSUPPORTED), ((1, (1 << 20) + 1, 8), UNSUPPORTED),
                            ((1, 8, (1 << 20) + 1), UNSUPPORTED),
                            ((65535, 1 << 20, 1 << 20), UNSUPPORTED)]:
        assert size(query, B, m, n)[0] == want, (B, m, n)
        assert _ortho(lib, B=B, m=m, n=n) == want
    assert query(1, 8, 8, None) == INVALID
    assert size(query, 0, 8, 8) == (OK, 0)
    assert _ortho(lib, B=0, x=None, out=None, ws=None, wsb=0) == OK
    assert _ortho(lib, dt=2) == UNSUPPORTED and _ortho(lib, odt=2) == UNSUPPORTED
    assert _ortho(lib, steps=-1) == INVALID and _ortho(lib, steps=65) == INVALID
    for eps in (-1.0, float("nan"), float("inf")):
        assert _ortho(lib, eps=eps) == INVALID
    for name in ("a", "b", "c"):
        assert _ortho(lib, **{name: float("nan")}) == INVALID
        assert _ortho(lib, **{name: float("inf")}) == INVALID
        assert _ortho(lib, **{name: 1e30}) == UNSUPPORTED
    assert _ortho(lib, a=50.0) == UNSUPPORTED                 # the iterate grows without end
    assert _ortho(lib, a=1.0, b=1.0, c=1e-3) == UNSUPPORTED   # b^2 > 64 |c|
    assert _ortho(lib, xs=64 * 128 - 4) == INVALID
    assert _ortho(lib, os_=64 * 128 - 4) == INVALID
    assert _ortho(lib, xs=64 * 128 + 2) == ALIGNMENT
    assert _ortho(lib, odt=1, os_=64 * 128 + 4) == ALIGNMENT
    for name in ("x", "out", "ws"):
        assert _ortho(lib, **{name: None}) == INVALID, name
        assert _ortho(lib, **{name: (1 << 38) + 8}) == ALIGNMENT, name
    for B, m, n in ((2, 64, 128), (1, 300, 500)):
        need = size(query, B, m, n)[1]
        assert need > 0
        assert _ortho(lib, B=B, m=m, n=n, xs=m * n, os_=m * n, wsb=need - 1) == WORKSPACE
    # x and out are one tensor with one layout, or do not touch
    assert _ortho(lib, out=1 << 30, odt=1) == INVALID
    assert _ortho(lib, out=1 << 30, os_=64 * 128 + 64) == INVALID
    assert _ortho(lib, out=(1 << 30) + 64 * 128 * 4) == INVALID
    assert _ortho(lib, ws=1 << 30) == INVALID and _ortho(lib, ws=1 << 34) == INVALID
    assert _ortho(lib, out=1 << 30, ws=(1 << 30) + 16) == INVALID


# ---------------------------------------------------------------- binding
def test_binding_refuses_wrong_tensors():
    x, w, off = torch.zeros(4, 8), torch.zeros(2, 6, 8), torch.zeros(3, dtype=torch.int32)
    stat = torch.zeros(4)
    for call in (
        lambda: mx.layer_norm(x),
        lambda: mx.layer_norm(x[0]),
        lambda: mx.layer_norm(x.double()),
        lambda: mx.layer_norm(x, torch.zeros(7)),
        lambda: mx.layer_norm(x, torch.zeros(8, dtype=torch.bfloat16)),
        lambda: mx.layer_norm(x, out=torch.zeros(4, 7)),
        lambda: mx.layer_norm_backward(x, x, None, stat, stat),
        lambda: mx.layer_norm_backward(x[:3], x, None, stat, stat),
        lambda: mx.layer_norm_backward(x, x, None, stat.double(), stat),
        lambda: mx.grouped_matmul(x, w, off),
        lambda: mx.grouped_matmul(x, torch.zeros(2, 6, 9), off),
        lambda: mx.grouped_matmul(x, w[0], off),
        lambda: mx.grouped_matmul(x, w, off[:2]),
        lambda: mx.grouped_matmul(x, w, off.long()),
        lambda: mx.grouped_matmul(x, w.to(torch.bfloat16), off),
        lambda: mx.grouped_matmul(x, w, off, out=torch.zeros(4, 5)),
        lambda: mx.grouped_matmul_backward(x, w, off, torch.zeros(4, 6)),
        lambda: mx.grouped_matmul_backward(x, w, off, torch.zeros(4, 5)),
        lambda: mx.orthogonalize(x),
        lambda: mx.orthogonalize(x[0]),
        lambda: mx.orthogonalize(x.half()),
    ):
        with pytest.raises(mx.MoEError):
            call()


def test_binding_refuses_sizes_past_int():
    """A size that the ABI's int would wrap around (here to 5) is refused, not shortened."""
    wide = (1 << 32) + 5
    x = torch.empty(wide, 8, device="meta")
    w, off = torch.empty(2, 6, 8, device="meta"), torch.empty(3, dtype=torch.int32, device="meta")
    stat = torch.empty(wide, device="meta")
    for call in (lambda: mx.layer_norm(x), lambda: mx.layer_norm_backward(x, x, None, stat, stat),
                 lambda: mx.grouped_matmul(x, w, off),
                 lambda: mx.grouped_matmul_backward(x, w, off, torch.empty(wide, 6, device="meta")),
                 lambda: mx.orthogonalize(x), lambda: mx.orthogonalize(torch.empty(1 << 17, 1 << 16, 2, 2, device="meta"))):
        with pytest.raises(mx.MoEError, match="2\\^31"):
            call()
