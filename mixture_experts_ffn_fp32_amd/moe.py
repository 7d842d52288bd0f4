"""Python binding of libmoe.so (ctypes): argument marshalling only.

Every step of the layer runs in the library's HIP kernels; PyTorch is used
here only to hold device memory and to name the current stream.  If the
library is missing, every call raises MoEError -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

LIB_PATH = os.environ.get("MOE_LIB_PATH") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_DTYPE_F32, MOE_DTYPE_BF16 = 0, 1
NUM_STAGES = 7
STAGE_NAMES = ("router", "tile_rank", "dispatch_scan", "scatter", "expert_gemm1_swiglu",
               "expert_gemm2_down", "combine")
MOE_DTYPE_E4M3, MOE_DTYPE_E5M2 = 2, 3
_DTYPES = {torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16}
_F8 = {torch.float8_e4m3fn: MOE_DTYPE_E4M3, torch.float8_e5m2: MOE_DTYPE_E5M2}

EXPORTED = ("moe_last_error", "moe_workspace_size", "moe_layer_forward",
            "moe_layer_forward_static", "moe_route",
            "moe_dispatch_workspace_size", "moe_dispatch", "moe_expert_ffn_workspace_size",
            "moe_expert_ffn", "moe_combine", "moe_balance_workspace_size", "moe_balance_stats",
            "moe_backward_workspace_size", "moe_layer_backward", "moe_layer_backward_aux",
            "moe_layer_norm",
            "moe_layer_norm_backward_workspace_size", "moe_layer_norm_backward",
            "moe_grouped_matmul_workspace_size", "moe_grouped_matmul",
            "moe_grouped_matmul_backward_workspace_size", "moe_grouped_matmul_backward",
            "moe_orthogonalize_workspace_size", "moe_orthogonalize", "moe_rms_norm",
            "moe_rms_norm_backward_workspace_size", "moe_rms_norm_backward", "moe_quantize_rows",
            "moe_quantize_blocks", "moe_dequantize_rows",
            "moe_grouped_matmul_quantized_workspace_size", "moe_grouped_matmul_quantized",
            "moe_grouped_matmul_quantized_dx_workspace_size", "moe_grouped_matmul_quantized_dx",
            "moe_balance_loss_workspace_size", "moe_balance_loss", "moe_balance_loss_backward",
            "moe_timing_enable", "moe_timing_read", "moe_timing_stages")


class MoEError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"moe status {status}: {message}")
        self.status = status
        self.message = message


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libmoe.so and declare its C signatures (loading needs no GPU)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise MoEError(-1, f"{path} is not built (python -m mixture_experts_ffn_fp32_amd.build)")
    L = ctypes.CDLL(path)
    vp, i, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    szp = ctypes.POINTER(ctypes.c_size_t)
    fl, i64 = ctypes.c_float, ctypes.c_int64
    L.moe_last_error.restype = ctypes.c_char_p
    L.moe_last_error.argtypes = []
    sigs = {
        "moe_workspace_size": [i, i, i, i, i, i, i, szp],
        "moe_layer_forward": [vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, vp, sz, vp],
        "moe_layer_forward_static": [vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, vp],
        "moe_route": [vp, vp, f, i, i, i, i, i, vp, vp, vp, vp],
        "moe_dispatch_workspace_size": [i, i, i, szp],
        "moe_dispatch": [vp, i, i, i, vp, vp, vp, vp, sz, vp],
        "moe_expert_ffn_workspace_size": [i, i, i, i, szp],
        "moe_expert_ffn": [vp, vp, vp, i, i, i, i, i, i, i, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_combine": [vp, vp, vp, i, i, i, i, i, vp, vp],
        "moe_balance_workspace_size": [i, i, szp],
        "moe_balance_stats": [vp, vp, i, i, i, vp, i, ctypes.c_float, ctypes.c_float, vp, vp, vp,
                              vp, vp, vp, sz, vp],
        "moe_backward_workspace_size": [i, i, i, i, i, i, i, szp],
        "moe_layer_backward": [vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, vp, vp, vp, vp, vp, vp,
                               sz, vp],
        "moe_layer_backward_aux": [vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, vp, vp, vp, vp, vp,
                                   vp, vp, sz, vp],
        "moe_layer_norm": [vp, vp, vp, i, i, fl, i, vp, vp, vp, vp],
        "moe_layer_norm_backward_workspace_size": [i, i, i, szp],
        "moe_layer_norm_backward": [vp, vp, vp, vp, vp, i, i, i, vp, vp, vp, vp, sz, vp],
        "moe_grouped_matmul_workspace_size": [i, i, i, i, i, szp],
        "moe_grouped_matmul": [vp, vp, vp, i, i, i, i, i, i, vp, vp, sz, vp],
        "moe_grouped_matmul_backward_workspace_size": [i, i, i, i, i, i, i, szp],
        "moe_grouped_matmul_backward": [vp, vp, vp, vp, i, i, i, i, i, i, vp, vp, vp, sz, vp],
        "moe_orthogonalize_workspace_size": [i, i, i, szp],
        "moe_orthogonalize": [vp, i64, i, i, i, i, i, fl, fl, fl, fl, vp, i64, i, vp, sz, vp],
        "moe_rms_norm": [vp, vp, vp, i, i, fl, i, i, vp, vp, vp, vp, vp],
        "moe_rms_norm_backward_workspace_size": [i, i, i, szp],
        "moe_rms_norm_backward": [vp, vp, vp, vp, vp, i, i, i, vp, vp, vp, sz, vp],
        "moe_quantize_rows": [vp, i, i, i, i, vp, vp, vp],
        "moe_quantize_blocks": [vp, i, i, i, i, i, vp, vp, vp],
        "moe_dequantize_rows": [vp, vp, i, i, i, i, vp, vp],
        "moe_grouped_matmul_quantized_workspace_size": [i, i, i, i, szp],
        "moe_grouped_matmul_quantized": [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, vp, sz, vp],
        "moe_grouped_matmul_quantized_dx_workspace_size": [i, i, i, i, szp],
        "moe_grouped_matmul_quantized_dx": [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, vp, sz, vp],
        "moe_balance_loss_workspace_size": [i, i, i, szp],
        "moe_balance_loss": [vp, vp, vp, vp, vp, i, i, i, i, i, fl, fl, vp, vp, vp, vp, vp, sz, vp],
        "moe_balance_loss_backward": [vp, vp, vp, vp, vp, i, i, i, vp, vp],
        "moe_timing_enable": [i],
        "moe_timing_read": [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int)],
        "moe_timing_stages": [ctypes.c_uint],
    }
    for name, args in sigs.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    _lib = L
    return L


def _check(status: int):
    if status != 0:
        raise MoEError(status, load_library().moe_last_error().decode())


def _p(t):
    return None if t is None else t.data_ptr()


def _dev(*tensors, dtype=None):
    """Every tensor must live on a GPU, be contiguous and (if given) of dtype."""
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise MoEError(1, "tensors must be on a GPU device")
        if not t.is_contiguous():
            raise MoEError(1, "tensors must be contiguous")
        if dtype is not None and t.dtype != dtype:
            raise MoEError(1, f"expected dtype {dtype}, got {t.dtype}")


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dtype_code(t) -> int:
    if t.dtype not in _DTYPES:
        raise MoEError(2, f"unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def _infer_I(W_routed, N: int, d: int) -> int:
    n = W_routed.numel()
    if N <= 0 or d <= 0 or n % (3 * N * d) != 0:
        raise MoEError(1, "W_routed must hold N blocks of 3*I*d elements")
    return n // (3 * N * d)


def workspace_size(T, d, I, N, K, K_s, dtype_code) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().moe_workspace_size(T, d, I, N, K, K_s, dtype_code, ctypes.byref(out)))
    return out.value


def layer_forward(u, E_gate, W_routed, W_shared, N: int, K: int, K_s: int, gate_bias=None,
                  out=None, workspace=None):
    """h = u + sum_shared FFN(u) + sum_topK g FFN(u); see include/moe.h."""
    L = load_library()
    T, d = u.shape
    dt = _dtype_code(u)
    _dev(u, E_gate, W_routed, W_shared, dtype=u.dtype)
    _dev(gate_bias, dtype=torch.float32)
    I = _infer_I(W_routed, N, d)
    h = torch.empty_like(u) if out is None else out
    _dev(h, dtype=u.dtype)
    need = workspace_size(T, d, I, N, K, K_s, dt)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=u.device)
    _dev(workspace)
    _check(L.moe_layer_forward(_p(u), _p(E_gate), _p(W_routed), _p(W_shared), N, K, K_s, T, d, I,
                               dt, _p(gate_bias), _p(h), _p(workspace),
                               workspace.numel() * workspace.element_size(), _stream()))
    return h


def layer_forward_static(u, E_gate, W_routed, W_shared, N: int, K: int, K_s: int,
                         gate_bias=None, out=None):
    """The layer forward with the library's static device scratch as its workspace (no
    device allocation inside the call; `out` may be given so that none is made here
    either).  Shapes needing more than MOE_STATIC_SCRATCH_BYTES raise MoEError."""
    L = load_library()
    T, d = u.shape
    dt = _dtype_code(u)
    _dev(u, E_gate, W_routed, W_shared, dtype=u.dtype)
    _dev(gate_bias, dtype=torch.float32)
    I = _infer_I(W_routed, N, d)
    h = torch.empty_like(u) if out is None else out
    _dev(h, dtype=u.dtype)
    _check(L.moe_layer_forward_static(_p(u), _p(E_gate), _p(W_routed), _p(W_shared), N, K, K_s,
                                      T, d, I, dt, _p(gate_bias), _p(h), _stream()))
    return h


def backward_workspace_size(T, d, I, N, K, K_s, dtype_code) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().moe_backward_workspace_size(T, d, I, N, K, K_s, dtype_code,
                                                      ctypes.byref(out)))
    return out.value


def layer_backward(u, E_gate, W_routed, W_shared, N: int, K: int, K_s: int, dh, gate_bias=None,
                   workspace=None, dlogits=None):
    """Gradients of sum(dh * h) for h = layer_forward(u, ...); see include/moe.h.

    dlogits [T][N] float32 (balance_loss_backward's) is the logits' gradient from losses
    beside h, and joins du, dE_gate and dgate_bias.

    Returns (du, dE_gate, dgate_bias, dW_routed, dW_shared or None); every gradient
    but du is float32, the weight gradients in the layout of their weights.  The
    bias gradient is the same whether or not a bias is given.
    """
    L = load_library()
    T, d = u.shape
    dt = _dtype_code(u)
    _dev(u, E_gate, W_routed, W_shared, dh, dtype=u.dtype)
    _dev(gate_bias, dlogits, dtype=torch.float32)
    if dlogits is not None:
        _typed("dlogits", dlogits, torch.float32, (T, N))
    I = _infer_I(W_routed, N, d)
    dev = u.device
    # an empty batch writes nothing: its weight gradients are zeros
    alloc = torch.zeros if T == 0 else torch.empty
    du = torch.empty_like(u)
    dE = alloc(E_gate.shape, dtype=torch.float32, device=dev)
    db = alloc(N, dtype=torch.float32, device=dev)
    dWr = alloc(W_routed.shape, dtype=torch.float32, device=dev)
    dWs = None if K_s == 0 else alloc(W_shared.shape, dtype=torch.float32, device=dev)
    need = backward_workspace_size(T, d, I, N, K, K_s, dt)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(workspace)
    _check(L.moe_layer_backward_aux(_p(u), _p(E_gate), _p(W_routed), _p(W_shared), N, K, K_s, T, d,
                                    I, dt, _p(gate_bias), _p(dh), _p(dlogits), _p(du), _p(dE),
                                    _p(db), _p(dWr), _p(dWs), _p(workspace),
                                    workspace.numel() * workspace.element_size(), _stream()))
    return du, dE, db, dWr, dWs


def route(u, E_gate, K: int, gate_bias=None, want_scores: bool = False):
    """(idx [T][K] int32, gate [T][K] float32, scores [T][N] float32 or None)."""
    L = load_library()
    T, d = u.shape
    N = E_gate.shape[0]
    _dev(u, E_gate, dtype=u.dtype)
    _dev(gate_bias, dtype=torch.float32)
    idx = torch.empty((T, K), dtype=torch.int32, device=u.device)
    gate = torch.empty((T, K), dtype=torch.float32, device=u.device)
    scores = torch.empty((T, N), dtype=torch.float32, device=u.device) if want_scores else None
    _check(L.moe_route(_p(u), _p(E_gate), _p(gate_bias), T, d, N, K, _dtype_code(u), _p(idx),
                       _p(gate), _p(scores), _stream()))
    return idx, gate, scores


def dispatch(idx, N: int):
    """(counts [N], offsets [N+1], sorted_pair [T*K]) int32, grouped by expert, stable."""
    L = load_library()
    T, K = idx.shape
    _dev(idx, dtype=torch.int32)
    out = ctypes.c_size_t(0)
    _check(L.moe_dispatch_workspace_size(T, N, K, ctypes.byref(out)))
    ws = torch.empty(max(out.value, 1), dtype=torch.uint8, device=idx.device)
    counts = torch.empty(N, dtype=torch.int32, device=idx.device)
    offsets = torch.empty(N + 1, dtype=torch.int32, device=idx.device)
    sorted_pair = torch.empty(max(T * K, 1), dtype=torch.int32, device=idx.device)
    _check(L.moe_dispatch(_p(idx), T, N, K, _p(counts), _p(offsets), _p(sorted_pair), _p(ws),
                          ws.numel(), _stream()))
    return counts, offsets, sorted_pair[:T * K]


def expert_ffn(u, W_routed, W_shared, N: int, K: int, K_s: int, offsets, sorted_pair, gate):
    """(H_routed [T*K][I], H_shared [T][K_s*I] or None, Y [T*K][d], Y_shared [T][d] or None)."""
    L = load_library()
    T, d = u.shape
    dt = _dtype_code(u)
    _dev(u, W_routed, W_shared, dtype=u.dtype)
    _dev(offsets, sorted_pair, dtype=torch.int32)
    _dev(gate, dtype=torch.float32)
    I = _infer_I(W_routed, N, d)
    out = ctypes.c_size_t(0)
    _check(L.moe_expert_ffn_workspace_size(T, N, K, K_s, ctypes.byref(out)))
    ws = torch.empty(max(out.value, 1), dtype=torch.uint8, device=u.device)
    H = torch.empty((T * K, I), dtype=u.dtype, device=u.device)
    Y = torch.empty((T * K, d), dtype=u.dtype, device=u.device)
    Hs = torch.empty((T, K_s * I), dtype=u.dtype, device=u.device) if K_s > 0 else None
    Ys = torch.empty((T, d), dtype=u.dtype, device=u.device) if K_s > 0 else None
    _check(L.moe_expert_ffn(_p(u), _p(W_routed), _p(W_shared), T, d, I, N, K, K_s, dt,
                            _p(offsets), _p(sorted_pair), _p(gate), _p(H), _p(Hs), _p(Y), _p(Ys),
                            _p(ws), ws.numel(), _stream()))
    return H, Hs, Y, Ys


def combine(u, Y, Y_shared, K: int, K_s: int):
    """h = u + Y_shared + sum_k Y[t*K+k]."""
    L = load_library()
    T, d = u.shape
    _dev(u, Y, Y_shared, dtype=u.dtype)
    h = torch.empty_like(u)
    _check(L.moe_combine(_p(u), _p(Y), _p(Y_shared), T, d, K, K_s, _dtype_code(u), _p(h),
                         _stream()))
    return h


def balance_stats(scores, idx, K: int, group_of=None, alpha1: float = 1.0, alpha2: float = 1.0):
    """Balance statistics of one batch: dict of f [N], P [N], L_ExpBal and, with
    group_of (a length-N sequence of device-group ids 0..D-1), f_dev [D],
    P_dev [D], L_DevBal.  Tensors are float32 on the scores' device."""
    L = load_library()
    T, N = scores.shape
    _dev(scores, dtype=torch.float32)
    _dev(idx, dtype=torch.int32)
    if idx.shape != (T, K):
        raise MoEError(1, "idx must be [T][K]")
    D = 0
    groups = None
    if group_of is not None:
        g = [int(x) for x in group_of]
        if len(g) != N:
            raise MoEError(1, "group_of must have N entries")
        D = max(g) + 1 if g else 0
        groups = (ctypes.c_int32 * N)(*g)
    out = ctypes.c_size_t(0)
    _check(L.moe_balance_workspace_size(T, N, ctypes.byref(out)))
    dev = scores.device
    ws = torch.empty(max(out.value, 1), dtype=torch.uint8, device=dev)
    f = torch.empty(N, dtype=torch.float32, device=dev)
    P = torch.empty(N, dtype=torch.float32, device=dev)
    fd = torch.empty(max(D, 1), dtype=torch.float32, device=dev)
    Pd = torch.empty(max(D, 1), dtype=torch.float32, device=dev)
    losses = torch.empty(2, dtype=torch.float32, device=dev)
    _check(L.moe_balance_stats(_p(scores), _p(idx), T, N, K, groups, D, alpha1, alpha2, _p(f),
                               _p(P), _p(fd), _p(Pd), _p(losses), _p(ws), ws.numel(), _stream()))
    res = {"f": f, "P": P, "L_ExpBal": losses[0]}
    if group_of is not None:
        res.update({"f_dev": fd[:D], "P_dev": Pd[:D], "L_DevBal": losses[1]})
    return res


# ---------------------------------------------------------------- operators beside the layer
# A call on a few rows takes about as long as the host needs for it, so the calls below avoid
# what costs microseconds: torch.cuda.current_stream() builds a Stream object (2.6 us; the raw
# handle takes 0.1), and a device guard is only entered where the operands' device is not the
# current one.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _Same:
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_SAME = _Same()


def _on(device):
    """Context in which `device` is the current device."""
    return _SAME if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _stream_of(device):
    """The current stream of `device`."""
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _operands(first, *others):
    """Every tensor given is contiguous and on the device of the first; returns that device."""
    device = first.device
    if device.type != "cuda":
        raise MoEError(1, "tensors must be on a GPU device")
    if not first.is_contiguous():
        raise MoEError(1, "tensors must be contiguous")
    for t in others:
        if t is None:
            continue
        if t.device != device:
            raise MoEError(1, f"tensors on different devices: {device} and {t.device}")
        if not t.is_contiguous():
            raise MoEError(1, "tensors must be contiguous")
    return device


def _typed(name: str, t, dtype, shape):
    """t (if given) has this dtype and shape."""
    if t is None:
        return
    if t.dtype != dtype:
        raise MoEError(1, f"{name}: expected dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise MoEError(1, f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


INT_MAX = 2 ** 31 - 1


def _dims(name: str, t, n: int):
    if t.dim() != n:
        raise MoEError(1, f"{name} must have {n} dimensions, got {t.dim()}")
    if max(t.shape) > INT_MAX:             # the ABI's sizes are int
        raise MoEError(2, f"{name}: sizes past 2^31 - 1 are not supported, got {tuple(t.shape)}")
    return t.shape


def _scratch(workspace, need: int, device):
    """The caller's workspace if it is large enough, else a new one (None: none needed).
    A new one comes from PyTorch's allocator for the current stream, like the outputs."""
    if workspace is not None:
        if _operands(workspace) != device:
            raise MoEError(1, f"workspace is on {workspace.device}, the operands on {device}")
        if workspace.numel() * workspace.element_size() >= need:
            return workspace
    return torch.empty(need, dtype=torch.uint8, device=device) if need > 0 else None


def _bytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _size(query, *args) -> int:
    out = ctypes.c_size_t(0)
    _check(query(*args, ctypes.byref(out)))
    return out.value


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None):
    """(y, mean, rstd) of layer norm over the last dimension of x [T][d]; see include/moe.h.

    weight and bias [d] have x's dtype (None: ones, zeros); mean and rstd [T] are float32,
    what layer_norm_backward needs."""
    L = load_library()
    T, d = _dims("x", x, 2)
    dt = _dtype_code(x)
    _typed("weight", weight, x.dtype, (d,))
    _typed("bias", bias, x.dtype, (d,))
    _typed("out", out, x.dtype, (T, d))
    dev = _operands(x, weight, bias, out)
    with _on(dev):
        y = torch.empty_like(x) if out is None else out
        mean = torch.empty(T, dtype=torch.float32, device=dev)
        rstd = torch.empty(T, dtype=torch.float32, device=dev)
        _check(L.moe_layer_norm(_p(x), _p(weight), _p(bias), T, d, eps, dt, _p(y), _p(mean),
                                _p(rstd), _stream_of(dev)))
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, workspace=None):
    """(dx, dweight, dbias) of sum(dy * y) for y, mean, rstd = layer_norm(x, weight, ..);
    dx has x's dtype, dweight and dbias [d] are float32.  weight may be None (ones)."""
    L = load_library()
    T, d = _dims("x", x, 2)
    dt = _dtype_code(x)
    _typed("dy", dy, x.dtype, (T, d))
    _typed("weight", weight, x.dtype, (d,))
    _typed("mean", mean, torch.float32, (T,))
    _typed("rstd", rstd, torch.float32, (T,))
    dev = _operands(x, dy, weight, mean, rstd)
    with _on(dev):
        dx = torch.empty_like(x)
        dw = torch.empty(d, dtype=torch.float32, device=dev)
        db = torch.empty(d, dtype=torch.float32, device=dev)
        ws = _scratch(workspace, _size(L.moe_layer_norm_backward_workspace_size, T, d, dt), dev)
        _check(L.moe_layer_norm_backward(_p(dy), _p(x), _p(weight), _p(mean), _p(rstd), T, d, dt,
                                         _p(dx), _p(dw), _p(db), _p(ws), _bytes(ws), _stream_of(dev)))
    return dx, dw, db


def _grouped_shapes(x, w, offsets):
    M, k = _dims("x", x, 2)
    E, n, kw = _dims("w", w, 3)
    if kw != k:
        raise MoEError(1, f"x has rows of {k}, w of {kw}")
    _typed("w", w, x.dtype, (E, n, k))
    _typed("offsets", offsets, torch.int32, (E + 1,))
    return M, E, n, k


def grouped_matmul(x, w, offsets, out=None, workspace=None):
    """y [M][n]: y[r] = w[e] @ x[r] for the rows offsets[e] <= r < offsets[e+1] of each group e.

    x [M][k], w [E][n][k] of one dtype, offsets [E+1] int32 on the device (dispatch()'s, or any
    non-decreasing ones).  Rows outside every group are zero in a new y and left as they were
    in a given `out`."""
    L = load_library()
    M, E, n, k = _grouped_shapes(x, w, offsets)
    dt = _dtype_code(x)
    _typed("out", out, x.dtype, (M, n))
    dev = _operands(x, w, offsets, out)
    with _on(dev):
        y = torch.empty((M, n), dtype=x.dtype, device=dev) if out is None else out
        ws = _scratch(workspace, _size(L.moe_grouped_matmul_workspace_size, M, E, n, k, dt), dev)
        _check(L.moe_grouped_matmul(_p(x), _p(w), _p(offsets), M, E, n, k, dt,
                                    1 if out is None else 0, _p(y), _p(ws), _bytes(ws),
                                    _stream_of(dev)))
    return y


def grouped_matmul_backward(x, w, offsets, dy, need_dx: bool = True, need_dw: bool = True,
                            workspace=None):
    """(dx, dw) of sum(dy * y) for y = grouped_matmul(x, w, offsets): dx [M][k] in x's dtype
    (zero outside the groups), dw [E][n][k] float32 (zero for a group without rows).  One that
    is not needed is None."""
    L = load_library()
    M, E, n, k = _grouped_shapes(x, w, offsets)
    dt = _dtype_code(x)
    _typed("dy", dy, x.dtype, (M, n))
    dev = _operands(x, w, offsets, dy)
    with _on(dev):
        dx = torch.empty_like(x) if need_dx else None
        dw = torch.empty((E, n, k), dtype=torch.float32, device=dev) if need_dw else None
        ws = _scratch(workspace, _size(L.moe_grouped_matmul_backward_workspace_size, M, E, n, k,
                                       dt, int(need_dx), int(need_dw)), dev)
        _check(L.moe_grouped_matmul_backward(_p(x), _p(w), _p(offsets), _p(dy), M, E, n, k, dt, 1,
                                             _p(dx), _p(dw), _p(ws), _bytes(ws), _stream_of(dev)))
    return dx, dw


def _matrices(name: str, t):
    """(batch, m, n, elements from one matrix to the next) of t [..][m][n]: contiguous, or
    [B][m][n] with contiguous matrices at a larger stride (the blocks of a weight gradient)."""
    if t.dim() < 2:
        raise MoEError(1, f"{name} must have at least 2 dimensions")
    m, n = t.shape[-2:]
    B = 1
    for s in t.shape[:-2]:
        B *= s
    if max(B, m, n) > INT_MAX:
        raise MoEError(2, f"{name}: sizes past 2^31 - 1 are not supported, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise MoEError(1, "tensors must be on a GPU device")
    if t.is_contiguous():
        return B, m, n, m * n
    if t.dim() != 3 or not t[0].is_contiguous() or t.stride(0) < m * n:
        raise MoEError(1, f"{name} must hold contiguous matrices, back to back or at one stride")
    return B, m, n, t.stride(0)


def orthogonalize(x, steps: int = 5, eps: float = 1e-7,
                  coefficients=(3.4445, -4.7750, 2.0315), out=None, out_dtype=None,
                  workspace=None):
    """The orthogonalised update of each matrix of x [..][m][n] (see include/moe.h): its
    Newton-Schulz iterate after `steps` steps, in out_dtype (default x's dtype).

    Takes gradients where they lie: x may be a view like layer_backward's
    dW_routed.view(N, 3, I * d)[:, 2].view(N, d, I), whose matrices are contiguous at one
    stride.  out may be x."""
    L = load_library()
    dt = _dtype_code(x)
    B, m, n, xs = _matrices("x", x)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype if out_dtype is None else out_dtype,
                          device=x.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise MoEError(1, f"out: expected dtype {out_dtype}, got {out.dtype}")
    if out.shape != x.shape:
        raise MoEError(1, f"out: expected shape {tuple(x.shape)}, got {tuple(out.shape)}")
    if out.device != x.device:
        raise MoEError(1, f"tensors on different devices: {x.device} and {out.device}")
    os_ = _matrices("out", out)[3]
    a, b, c = (float(v) for v in coefficients)
    with _on(x.device):
        ws = _scratch(workspace, _size(L.moe_orthogonalize_workspace_size, B, m, n), x.device)
        _check(L.moe_orthogonalize(_p(x), xs, B, m, n, dt, steps, eps, a, b, c, _p(out), os_,
                                   _dtype_code(out), _p(ws), _bytes(ws), _stream_of(x.device)))
    return out


# ---------------------------------------------------------------- experts in 8 bits
F8_BLOCK = 128


def _f8_code(name: str, dtype) -> int:
    if dtype not in _F8:
        raise MoEError(2, f"{name}: expected torch.float8_e4m3fn or torch.float8_e5m2, got {dtype}")
    return _F8[dtype]


def _f8_blocks(n: int) -> int:
    return (n + F8_BLOCK - 1) // F8_BLOCK


def _rms_norm(x, weight, residual, eps, q_dtype, h_out, out):
    L = load_library()
    T, d = _dims("x", x, 2)
    dt = _dtype_code(x)
    yt = dt if q_dtype is None else _f8_code("q_dtype", q_dtype)
    _typed("weight", weight, x.dtype, (d,))
    _typed("residual", residual, x.dtype, (T, d))
    _typed("h_out", h_out, x.dtype, (T, d))
    _typed("out", out, x.dtype if q_dtype is None else q_dtype, (T, d))
    dev = _operands(x, weight, residual, h_out, out)
    with _on(dev):
        h = h_out
        if h is None and residual is not None:
            h = torch.empty_like(x)
        y = torch.empty_like(x, dtype=q_dtype) if out is None else out
        scales = None
        if q_dtype is not None:
            scales = torch.empty((T, _f8_blocks(d)), dtype=torch.float32, device=dev)
        rstd = torch.empty(T, dtype=torch.float32, device=dev)
        _check(L.moe_rms_norm(_p(x), _p(residual), _p(weight), T, d, eps, dt, yt, _p(h), _p(y),
                              _p(scales), _p(rstd), _stream_of(dev)))
    return y, scales, x if h is None else h, rstd


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6, h_out=None, out=None):
    """(y, h, rstd): root-mean-square norm of h = x + residual over the last dimension of
    x [T][d] (see include/moe.h); without residual and h_out, h is x itself.

    weight [d] has x's dtype (None: ones), rstd [T] is float32; h and rstd are what
    rms_norm_backward needs.  h_out may be x or residual."""
    y, _, h, rstd = _rms_norm(x, weight, residual, eps, None, h_out, out)
    return y, h, rstd


def rms_norm_quantized(x, weight=None, residual=None, eps: float = 1e-6,
                       q_dtype=torch.float8_e4m3fn, h_out=None, out=None):
    """(q, scales, h, rstd): rms_norm with y in 8 bits, quantised as quantize_rows does from the
    float32 values: q [T][d] q_dtype, scales [T][ceil(d / 128)] float32."""
    return _rms_norm(x, weight, residual, eps, q_dtype, h_out, out)


def rms_norm_backward(dy, h, weight, rstd, dh=None, out=None, workspace=None):
    """(dx, dweight) of sum(dy * y) + sum(dh * h) for y, h, rstd = rms_norm(x, weight, residual):
    dx, of x and of residual alike, has h's dtype, dweight [d] is float32.  weight may be None
    (ones); dh, what reaches h from later layers, may be None; out may be dh."""
    L = load_library()
    T, d = _dims("h", h, 2)
    dt = _dtype_code(h)
    _typed("dy", dy, h.dtype, (T, d))
    _typed("weight", weight, h.dtype, (d,))
    _typed("rstd", rstd, torch.float32, (T,))
    _typed("dh", dh, h.dtype, (T, d))
    _typed("out", out, h.dtype, (T, d))
    dev = _operands(h, dy, weight, rstd, dh, out)
    with _on(dev):
        dx = torch.empty_like(h) if out is None else out
        dw = torch.empty(d, dtype=torch.float32, device=dev)
        ws = _scratch(workspace, _size(L.moe_rms_norm_backward_workspace_size, T, d, dt), dev)
        _check(L.moe_rms_norm_backward(_p(dy), _p(h), _p(weight), _p(rstd), _p(dh), T, d, dt,
                                       _p(dx), _p(dw), _p(ws), _bytes(ws), _stream_of(dev)))
    return dx, dw


def quantize_rows(x, q_dtype=torch.float8_e4m3fn):
    """(q, scales): x [T][d] in 8 bits with one float32 scale for each 128 columns of a row
    (see include/moe.h): q [T][d] q_dtype, scales [T][ceil(d / 128)]."""
    L = load_library()
    T, d = _dims("x", x, 2)
    dt, qt = _dtype_code(x), _f8_code("q_dtype", q_dtype)
    dev = _operands(x)
    with _on(dev):
        q = torch.empty_like(x, dtype=q_dtype)
        scales = torch.empty((T, _f8_blocks(d)), dtype=torch.float32, device=dev)
        _check(L.moe_quantize_rows(_p(x), T, d, dt, qt, _p(q), _p(scales), _stream_of(dev)))
    return q, scales


def quantize_blocks(w, q_dtype=torch.float8_e4m3fn):
    """(q, scales): matrices w [E][n][k] in 8 bits with one float32 scale for each 128 x 128:
    q [E][n][k] q_dtype, scales [E][ceil(n / 128)][ceil(k / 128)]."""
    L = load_library()
    E, n, k = _dims("w", w, 3)
    dt, qt = _dtype_code(w), _f8_code("q_dtype", q_dtype)
    dev = _operands(w)
    with _on(dev):
        q = torch.empty_like(w, dtype=q_dtype)
        scales = torch.empty((E, _f8_blocks(n), _f8_blocks(k)), dtype=torch.float32, device=dev)
        _check(L.moe_quantize_blocks(_p(w), E, n, k, dt, qt, _p(q), _p(scales), _stream_of(dev)))
    return q, scales


def dequantize_rows(q, scales, dtype=torch.bfloat16):
    """x [T][d] = q * scales in dtype, for q, scales = quantize_rows(..)."""
    L = load_library()
    T, d = _dims("q", q, 2)
    qt = _f8_code("q", q.dtype)
    if dtype not in _DTYPES:
        raise MoEError(2, f"unsupported dtype {dtype}")
    _typed("scales", scales, torch.float32, (T, _f8_blocks(d)))
    dev = _operands(q, scales)
    with _on(dev):
        x = torch.empty_like(q, dtype=dtype)
        _check(L.moe_dequantize_rows(_p(q), _p(scales), T, d, qt, _DTYPES[dtype], _p(x),
                                     _stream_of(dev)))
    return x


def _quantized(dx, x, xs, w, ws, offsets, out_dtype, out, workspace):
    L = load_library()
    name = "dy" if dx else "x"
    M, into = _dims(name, x, 2)
    E, n, k = _dims("w", w, 3)
    width = k if dx else n
    if into != (n if dx else k):
        raise MoEError(1, f"{name} has rows of {into}, w is {n} x {k}")
    code = _f8_code(name, x.dtype)
    if w.dtype != torch.float8_e4m3fn:
        raise MoEError(2, f"w: expected torch.float8_e4m3fn, got {w.dtype}")
    if out_dtype not in _DTYPES:
        raise MoEError(2, f"unsupported out_dtype {out_dtype}")
    _typed(name + "s", xs, torch.float32, (M, _f8_blocks(into)))
    _typed("ws", ws, torch.float32, (E, _f8_blocks(n), _f8_blocks(k)))
    if offsets is None and E != 1:
        raise MoEError(1, "offsets are needed where w holds more than one matrix")
    _typed("offsets", offsets, torch.int32, (E + 1,))
    _typed("out", out, out_dtype, (M, width))
    dev = _operands(x, xs, w, ws, offsets, out)
    size, call = ((L.moe_grouped_matmul_quantized_dx_workspace_size,
                   L.moe_grouped_matmul_quantized_dx) if dx else
                  (L.moe_grouped_matmul_quantized_workspace_size, L.moe_grouped_matmul_quantized))
    with _on(dev):
        y = torch.empty((M, width), dtype=out_dtype, device=dev) if out is None else out
        scratch = _scratch(workspace, _size(size, M, E, n, k), dev)
        _check(call(_p(x), _p(xs), _p(w), _p(ws), _p(offsets), M, E, n, k, code,
                    _DTYPES[out_dtype], 1 if out is None else 0, _p(y), _p(scratch),
                    _bytes(scratch), _stream_of(dev)))
    return y


def grouped_matmul_quantized(x, xs, w, ws, offsets=None, out_dtype=torch.bfloat16, out=None,
                             workspace=None):
    """y [M][n] in out_dtype: grouped_matmul of 8-bit rows and weights, x, xs = quantize_rows(..)
    (or rms_norm_quantized's), w, ws = quantize_blocks(..) in e4m3; see include/moe.h.

    offsets [E+1] as grouped_matmul's (None: all rows by the one matrix).  Rows outside every
    group are zero in a new y and left as they were in a given `out`."""
    return _quantized(False, x, xs, w, ws, offsets, out_dtype, out, workspace)


def grouped_matmul_quantized_dx(dy, dys, w, ws, offsets=None, out_dtype=torch.bfloat16, out=None,
                                workspace=None):
    """dx [M][k] in out_dtype: the rows' gradient of grouped_matmul_quantized for
    dy, dys = quantize_rows(dy [M][n], ..) and the forward's w, ws.  The weights' gradient is
    grouped_matmul_backward's, from rows in x's dtype (dequantize_rows reads them back)."""
    return _quantized(True, dy, dys, w, ws, offsets, out_dtype, out, workspace)


# ---------------------------------------------------------------- balance loss
def _sequences(T, offsets, mask):
    S = 1
    if offsets is not None:
        S = _dims("offsets", offsets, 1)[0] - 1
        _typed("offsets", offsets, torch.int32, (S + 1,))
    _typed("mask", mask, torch.bool, (T,))
    return S


def balance_loss(scores, idx, offsets=None, mask=None, device_of=None, devices: int = 0,
                 alpha1: float = 1.0, alpha2: float = 1.0, workspace=None):
    """The balance losses of a routed batch with what their gradient needs (see include/moe.h):
    a dict of counts [S][N] int32, P [S][N], losses [S][2] (expert-level, device-level) and
    slopes [S][2][N], float32.

    scores [T][N] and idx [T][K] are route()'s.  offsets [S+1] int32 cuts the rows into
    sequences with losses of their own (None: one), mask [T] bool says which rows count (None:
    all), device_of [N] int32 puts experts on `devices` devices (None: no device-level loss)."""
    L = load_library()
    T, N = _dims("scores", scores, 2)
    K = _dims("idx", idx, 2)[1]
    _typed("scores", scores, torch.float32, (T, N))
    _typed("idx", idx, torch.int32, (T, K))
    _typed("device_of", device_of, torch.int32, (N,))
    S = _sequences(T, offsets, mask)
    dev = _operands(scores, idx, offsets, mask, device_of)
    with _on(dev):
        counts = torch.empty((S, N), dtype=torch.int32, device=dev)
        P = torch.empty((S, N), dtype=torch.float32, device=dev)
        losses = torch.empty((S, 2), dtype=torch.float32, device=dev)
        slopes = torch.empty((S, 2, N), dtype=torch.float32, device=dev)
        ws = _scratch(workspace, _size(L.moe_balance_loss_workspace_size, T, N, S), dev)
        _check(L.moe_balance_loss(_p(scores), _p(idx), _p(offsets), _p(mask), _p(device_of), T, N,
                                  K, S, devices, alpha1, alpha2, _p(counts), _p(P), _p(losses),
                                  _p(slopes), _p(ws), _bytes(ws), _stream_of(dev)))
    return {"counts": counts, "P": P, "losses": losses, "slopes": slopes}


def balance_loss_backward(scores, slopes, dlosses=None, offsets=None, mask=None):
    """dlogits [T][N] float32: the gradient of sum(dlosses * losses) by the logits behind the
    scores, for slopes of balance_loss(scores, .., offsets, mask); dlosses [S][2] float32 (None:
    ones).  layer_backward takes it as `dlogits`."""
    L = load_library()
    T, N = _dims("scores", scores, 2)
    _typed("scores", scores, torch.float32, (T, N))
    S = _sequences(T, offsets, mask)
    _typed("slopes", slopes, torch.float32, (S, 2, N))
    _typed("dlosses", dlosses, torch.float32, (S, 2))
    dev = _operands(scores, slopes, dlosses, offsets, mask)
    with _on(dev):
        dlogits = torch.empty_like(scores)
        _check(L.moe_balance_loss_backward(_p(scores), _p(slopes), _p(dlosses), _p(offsets),
                                           _p(mask), T, N, S, _p(dlogits), _stream_of(dev)))
    return dlogits


def timing_enable(on: bool = True, stages=None):
    """Per-stage event timing on or off; `stages` (names) limits it to those stages."""
    L = load_library()
    mask = 0xFFFFFFFF if stages is None else sum(1 << STAGE_NAMES.index(s) for s in stages)
    _check(L.moe_timing_stages(mask))
    _check(L.moe_timing_enable(1 if on else 0))


def timing_read():
    """{stage name: (total ms, launches)} for the stage launches since the last read."""
    ms = (ctypes.c_double * NUM_STAGES)()
    n = (ctypes.c_int * NUM_STAGES)()
    _check(load_library().moe_timing_read(ms, n))
    return {STAGE_NAMES[i]: (ms[i], n[i]) for i in range(NUM_STAGES)}
