"""The 8-bit operators, the RMS norm and the balance loss at the ends of their ranges: tensors
past 4 GiB, the longest contractions, the most groups, infinities, two calls at once, padded
operands in graphs.  Tolerances as in test_gpu_quantized.py."""
import numpy as np
import pytest
import torch

from oracle import operators as ref
from parity_helpers import say
from test_gpu_quantized import (DT, F8, STORE, U, _balance_check, _product_check, _quantized, _ragged,
                                _routing, dev, host, ints, rounded, within)

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mixture_experts_ffn_fp32_amd")


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("M,E,n,k", [(3, 1, 2, 1 << 20), (3, 1, 1 << 20, 2), (2, 1, (1 << 20) - 3, 16),
                                     (2, 1, 17, (1 << 20) - 1), (1500, 1024, 130, 96), (5, 1024, 16, 16)])
def test_longest_rows_and_most_groups(M, E, n, k, dx):
    _product_check(M, E, n, k, _ragged(M, E, 7), dx, "e4m3", "f32", "ends of the range")
    _product_check(M, E, n, k, _ragged(M, E, 8), dx, "e5m2", "bf16", "ends of the range", 3)


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("length", [1, 15, 16, 17, 112, 127, 128, 129, 144, 240, 255, 256, 257, 272, 383, 384, 400])
def test_every_kind_of_tail(length, dx):
    """Contractions that end anywhere in a k-step, in every size of tile."""
    for M, width in ((3, 40), (700, 2080), (2100, 4112)):
        n, k = (length, width) if dx else (width, length)
        x, xs = _quantized((M, length), 5, "e4m3")
        w, ws = _quantized((1, n, k), 6, "e4m3", True)
        say(f"tail {length} dx={dx} M={M} width={width}")
        call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
        xv = host(x) * ref.spread_rows(host(xs), length)
        wv = (host(w) * ref.spread_matrix(host(ws), n, k))[0]
        want, size = (xv @ wv, abs(xv) @ abs(wv)) if dx else (xv @ wv.T, abs(xv) @ abs(wv).T)
        for out in ("f32", "bf16"):
            tol = (length + 16) * 2 * U * size + (2.0 ** -10 * size if out == "bf16" else 0)
            within(call(x, xs, w, ws, None, DT[out]), want, tol + STORE[out] * (np.abs(want) + tol), out)


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("M,E,n,k", [(200, 40, 601, 1001), (90, 30, 1409, 519), (64, 1, 17, 31), (1, 1, 16, 17),
                                     (7, 2, 31, 16), (30, 3, 2000, 2047), (130, 2, 515, 16), (640, 10, 517, 530)])
def test_odd_rows_read_in_place(M, E, n, k, dx):
    """Rows that start at any byte, few of them per group; every operand ends with its tensor."""
    off = _ragged(M, E, M)
    _product_check(M, E, n, k, off, dx, "e4m3", "f32", "in place")
    x, xs, w, ws, o, y = _product_check(M, E, n, k, off, dx, "e5m2", "bf16", "in place", 3)
    # what lies before and behind the operands in memory reaches no result
    call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized

    def inside(t):
        big = torch.full((t.numel() + 64,), 0x7f, dtype=torch.uint8, device="cuda")
        big[32:32 + t.numel()] = t.view(torch.uint8).reshape(-1)
        return big[32:32 + t.numel()].view(t.dtype).view(t.shape)

    assert torch.equal(call(inside(x), xs, inside(w), ws, o), y)


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("M,E,width", [(4096, 1, 4200), (4400, 3, 4000), (4500, 2, 3900), (5200, 4, 4200),
                                       (5700, 9, 4096), (6300, 5, 4004), (4100, 30, 1408)])
def test_last_rounds_of_few_tiles(M, E, width, dx):
    """One round of 256 x 256 tiles and some: the rest is cut to halves or quarters, some of which
    lie outside their group or the matrix.  A given out keeps the rows outside the groups."""
    n, k = (160, width) if dx else (width, 160)
    offsets = _ragged(M, E, M, 3)
    x, xs, w, ws, off, y = _product_check(M, E, n, k, offsets, dx, "e4m3", "bf16", "few tiles left")
    call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
    out = torch.full_like(y, 7.0)
    call(x, xs, w, ws, off, out=out)
    assert torch.equal(out[:offsets[-1]], y[:offsets[-1]]) and (out[offsets[-1]:] == 7).all()
    _product_check(M, E, n, k, offsets, dx, "e5m2", "bf16", "few tiles left", 1)


def test_product_of_rows_past_4_gib():
    """x past 2^32 bytes and, behind it, results: the last rows are as those of a small call."""
    M, n, k = (1 << 21) + 4096, 16, 2064
    assert M * k > 1 << 32
    say(f"rows past 4 GiB M={M}")
    x = torch.zeros((M, k), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    xs = torch.ones((M, 17), device="cuda")
    last, scales = _quantized((300, k), 1, "e4m3")
    w, ws = _quantized((2, n, k), 2, "e4m3", True)
    x.view(torch.uint8)[-300:] = last.view(torch.uint8)
    xs[-300:] = scales
    want, size = ref.grouped_matmul_quantized(host(last), host(scales), host(w)[1:], host(ws)[1:], [0, 300])
    for out in ("f32", "bf16"):
        y = mx.grouped_matmul_quantized(x, xs, w, ws, ints([0, M - 300, M]), DT[out])
        tol = (k + 32) * 2 * U * size + (2.0 ** -10 * size if out == "bf16" else 0)
        within(y[-300:], want, tol + STORE[out] * (np.abs(want) + tol), out)
        assert not y[:-300].any()


def test_weights_past_4_gib():
    E, n, k = 1030 // 2, 2064, 4112
    assert E * n * k > 1 << 32
    say(f"weights past 4 GiB E={E}")
    w = torch.zeros((E, n, k), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ws = torch.ones((E, 17, 33), device="cuda")
    last, scales = _quantized((1, n, k), 3, "e4m3", True)
    w.view(torch.uint8)[-1] = last.view(torch.uint8)[0]
    ws[-1] = scales[0]
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = 40
    for dx in (False, True):
        x, xs = _quantized((40, n if dx else k), 4, "e4m3")
        call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
        oracle = ref.grouped_matmul_quantized_dx if dx else ref.grouped_matmul_quantized
        want, size = oracle(host(x), host(xs), host(last), host(scales), [0, 40])
        for out in ("f32", "bf16"):
            tol = (x.shape[1] + 50) * 2 * U * size + (2.0 ** -10 * size if out == "bf16" else 0)
            within(call(x, xs, w, ws, off, DT[out]), want, tol + STORE[out] * (np.abs(want) + tol), out)


def test_rows_past_4_gib_in_the_memory_bound_operators():
    T, d = (1 << 20) + 77, 2056                     # 2.2e9 elements
    say(f"norm and quantising past 4 GiB T={T}")
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    r = np.random.default_rng(1)
    tail = dev(r.normal(size=(50, d)), "bf16")
    w = dev(1 + 0.1 * r.normal(size=d), "bf16")
    x[-50:] = tail
    q, s = mx.quantize_rows(x)
    q0, s0 = mx.quantize_rows(tail)
    assert torch.equal(q[-50:].view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s[-50:], s0)
    assert (s[:-50] == 1).all()
    assert torch.equal(mx.dequantize_rows(q, s)[-50:], mx.dequantize_rows(q0, s0))
    q, s, h, rstd = mx.rms_norm_quantized(x, w, x)
    q0, s0, h0, rstd0 = mx.rms_norm_quantized(tail, w, tail)
    assert torch.equal(q[-50:].view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s[-50:], s0)
    assert torch.equal(h[-50:], h0) and torch.equal(rstd[-50:], rstd0)
    del q, s
    dx, dw = mx.rms_norm_backward(x, h, w, rstd, x)
    dx0, dw0 = mx.rms_norm_backward(tail, h0, w, rstd0, tail)
    assert torch.equal(dx[-50:], dx0)
    size = (tail.double() * h0.double() * rstd0.double()[:, None]).abs().sum(0)
    assert ((dw - dw0).double().abs() <= 2 * (T + 12) * U * size).all()


def test_blocks_past_4_gib():
    E, n, k = 67, 8200, 8200                        # 4.5e9 elements
    say(f"quantize_blocks past 4 GiB E={E}")
    w = torch.zeros((E, n, k), dtype=torch.bfloat16, device="cuda")
    w[-1] = torch.randn(n, k, device="cuda").bfloat16()
    q, s = mx.quantize_blocks(w)
    q0, s0 = mx.quantize_blocks(w[-1:].contiguous())
    assert torch.equal(q[-1:].view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s[-1:], s0)
    assert (s[:-1] == 1).all() and not q[:3].view(torch.uint8).any()


def test_scores_past_4_gib():
    T, N = (1 << 22) + 1000, 256
    say(f"balance loss past 4 GiB T={T}")
    s, idx = _routing(1000, N, 4, 3)
    scores = torch.zeros((T, N), device="cuda")
    scores[-1000:] = dev(s)
    at = torch.zeros((T, 4), dtype=torch.int32, device="cuda")
    at[-1000:] = torch.from_numpy(idx).cuda()
    off = ints([0, T - 1000, T])
    b = mx.balance_loss(scores, at, off)
    c = mx.balance_loss(dev(s), torch.from_numpy(idx).cuda())
    assert torch.equal(b["counts"][1], c["counts"][0]) and torch.equal(b["P"][1], c["P"][0])
    assert torch.equal(b["slopes"][1], c["slopes"][0]) and int(b["counts"][0, 0]) == 4 * (T - 1000)
    z = mx.balance_loss_backward(scores, b["slopes"], None, off)
    assert torch.equal(z[-1000:], mx.balance_loss_backward(dev(s), c["slopes"])) and not z[:-1000].any()


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_infinities_of_e5m2_rows(out):
    M, n, k = 40, 160, 272
    x, xs = _quantized((M, k), 1, "e5m2")
    w, ws = _quantized((1, n, k), 2, "e4m3", True)
    y = mx.grouped_matmul_quantized(x, xs, w, ws, None, DT[out])
    x.view(torch.uint8)[7, 33] = 0x7c                       # + infinity
    w.view(torch.uint8)[0, 5, 33] = 0                       # times zero
    z = mx.grouped_matmul_quantized(x, xs, w, ws, None, DT[out])
    rest = torch.ones(M, n, dtype=torch.bool, device="cuda")
    rest[7], rest[:, 5] = False, False
    assert torch.equal(z[rest], y[rest])
    sign = torch.sign(w[0, :, 33].float())
    assert torch.isnan(z[7, 5]) and torch.equal(z[7].float().nan_to_num(0.0, np.inf, -np.inf)[sign != 0],
                                                (sign * np.inf)[sign != 0])


@pytest.mark.parametrize("M,E,n,k", [(600, 3, 270, 333), (5000, 3, 1030, 333)])
def test_two_calls_at_once(M, E, n, k):
    """The same operands on two streams, each call with a workspace of its own."""
    x, xs, w, ws, off, y = _product_check(M, E, n, k, _ragged(M, E, 1), False, "e4m3", "bf16", "one call")
    s, idx = _routing(3000, 64, 6, 1)
    s, idx = dev(s), torch.from_numpy(idx).cuda()
    b = mx.balance_loss(s, idx)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for st in streams:
            with torch.cuda.stream(st):
                got.append((mx.grouped_matmul_quantized(x, xs, w, ws, off), mx.balance_loss(s, idx)))
    torch.cuda.synchronize()
    for yy, bb in got:
        assert torch.equal(yy, y) and all(torch.equal(bb[i], b[i]) for i in b)


@pytest.mark.parametrize("M,E,n,k", [(300, 2, 136, 267), (9000, 2, 1100, 267)])
def test_odd_operands_in_a_graph(M, E, n, k):
    """Rows of no whole number of 16 bytes, read in place or copied to a workspace first: captured,
    replayed on new inputs with eager calls in between, two graphs with one workspace in turn."""
    ws_ = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    t = dict(zip(("x", "xs"), _quantized((M, k), 1, "e4m3")))
    t |= dict(zip(("w", "ws"), _quantized((E, n, k), 2, "e4m3", True)))
    t |= dict(zip(("dy", "dys"), _quantized((M, n), 3, "e5m2")), off=ints([0, M // 2 + 20, M]))

    def step(**kw):
        return [mx.grouped_matmul_quantized(t["x"], t["xs"], t["w"], t["ws"], t["off"], **kw),
                mx.grouped_matmul_quantized_dx(t["dy"], t["dys"], t["w"], t["ws"], t["off"], torch.float32,
                                               **kw)]

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(workspace=ws_)
        graphs.append((g, out))
    for i in range(4):
        for a, b, shape, seed, kind, m in (("x", "xs", (M, k), 10, "e4m3", False),
                                           ("w", "ws", (E, n, k), 20, "e4m3", True),
                                           ("dy", "dys", (M, n), 30, "e5m2", False)):
            q, s = _quantized(shape, seed + i, kind, m)
            t[a].view(torch.uint8).copy_(q.view(torch.uint8))
            t[b].copy_(s)
        want = step()
        g, out = graphs[i & 1]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_the_same_index_twice_and_one_sequence_of_every_row():
    s, idx = _routing(200, 40, 5, 2)
    idx[:, 1] = idx[:, 0]                                   # counted twice, as it stands twice
    _balance_check(s, idx, [0, 200], None, [0] * 40, 1, "the same index twice")
    _balance_check(s, idx, [0] + list(range(1, 201)), None, None, 0, "a sequence of each row")


def test_quantized_norm_is_the_norm_quantized():
    """The fused output agrees with quantising the float32 norm: the same float32 values."""
    r = np.random.default_rng(3)
    x, w = dev(r.normal(size=(77, 1000))), dev(1 + 0.1 * r.normal(size=1000))
    q, s, _, _ = mx.rms_norm_quantized(x, w)
    y = mx.rms_norm(x, w)[0]
    q2, s2 = mx.quantize_rows(y)
    assert torch.equal(s, s2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
    for kind, t in F8.items():
        rounded(mx.quantize_rows(y, t)[0], host(y) / ref.spread_rows(ref.block_scales(host(y), kind), 1000),
                4 * U, kind, kind)
