"""8-bit products and the norm's weight gradient on whole numbers and scales that are powers of two:
every product, cut-off sum and partial sum is exact in any order, so results equal the oracle's bit
for bit (rounded once where the storage type has fewer bits).  A value lost, doubled or taken from
another place shows, whatever the lengths are.  Also: results do not depend on other rows."""
import numpy as np
import pytest
import torch

from oracle import operators as ref
from parity_helpers import say
from test_gpu_quantized import DT, F8, STORE, _quantized, _ragged, dev, host, ints

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mixture_experts_ffn_fp32_amd")

# M, E, n, k.  bfloat16 results: 64^2 tiles, odd rows in place, 128^2, 256^2 (y or both), odd rows copied
# for 128^2 and 256^2, 256^2 with a last round in halves or quarters
SHAPES = [(3, 2, 7, 5), (40, 2, 144, 272), (70, 1, 130, 261), (300, 5, 320, 64), (700, 3, 1040, 1040),
          (2600, 3, 1536, 1408), (5000, 3, 2064, 2064), (6000, 3, 2064, 2064), (6100, 30, 1408, 2064),
          (5000, 2, 1030, 1037), (6000, 7, 2050, 2100), (4096, 1, 4200, 160), (5200, 4, 4208, 272),
          (6300, 5, 4004, 160), (4500, 2, 160, 3900), (6300, 5, 160, 4004), (7000, 3, 2064, 272),
          (12000, 2, 2064, 16), (2, 1, 30, 4111)]


def _whole(shape, seed, kind, matrices=False):
    """-2 .. 2, with scales of 1/2, 1 and 2: a block's sum is at most 512, a result at most 2^9 4 blocks,
    in quarters, which float32 holds exactly."""
    r = np.random.default_rng(seed)
    q = torch.from_numpy(r.integers(-2, 3, size=shape).astype(np.float32)).to(F8[kind]).cuda()
    s = (shape[0], -(-shape[1] // 128), -(-shape[2] // 128)) if matrices else (shape[0], -(-shape[1] // 128))
    return q, dev(np.exp2(r.integers(-1, 2, size=s)))


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("M,E,n,k", SHAPES)
def test_products_of_whole_numbers(M, E, n, k, dx, out, kind):
    say(f"whole numbers M={M} E={E} n={n} k={k} dx={dx} {kind} {out}")
    x, xs = _whole((M, n if dx else k), M + n, kind)
    w, ws = _whole((E, n, k), M + k, "e4m3", True)
    offsets = _ragged(M, E, M + E, M // 50)
    call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
    oracle = ref.grouped_matmul_quantized_dx if dx else ref.grouped_matmul_quantized
    want, size = oracle(host(x), host(xs), host(w), host(ws), offsets)
    assert size.max() * 4 < 2 ** 24
    want = torch.from_numpy(want).float().to(DT[out])       # exact, then one rounding
    for seed in range(2):                                   # twice: neither depends on what lay in y
        y = call(x, xs, w, ws, ints(offsets), DT[out], out=torch.full(want.shape, 7.0 + seed, dtype=DT[out],
                                                                      device="cuda"))
        rows = offsets[-1]
        wrong = (y[:rows].cpu() != want[:rows]).nonzero()
        assert len(wrong) == 0, (len(wrong), wrong[:5].tolist())
        assert (y[rows:] == 7.0 + seed).all()


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("M,E,n,k", [s for s in SHAPES if s[0] >= 2600])
def test_bfloat16_results_are_off_by_their_rounding(M, E, n, k, dx):
    """Values of every size: the norm of the error is that of the rounding itself (0.29 of a step in the
    mean, 1.7e-3 of the norm) and what the matrix instructions cut off (1.5e-5 of the norm)."""
    say(f"rounding M={M} E={E} n={n} k={k} dx={dx}")
    x, xs = _quantized((M, n if dx else k), 1, "e4m3")
    w, ws = _quantized((E, n, k), 2, "e4m3", True)
    offsets = _ragged(M, E, M)
    call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
    oracle = ref.grouped_matmul_quantized_dx if dx else ref.grouped_matmul_quantized
    want, _ = oracle(host(x), host(xs), host(w), host(ws), offsets)
    own = np.linalg.norm(host(torch.from_numpy(want).float().bfloat16()) - want)
    off_by = np.linalg.norm(host(call(x, xs, w, ws, ints(offsets))) - want)
    assert off_by <= 1.01 * own, off_by / own


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("M,E,n,k", [(40, 2, 144, 272), (70, 1, 130, 261), (700, 3, 1040, 1040), (5000, 2, 1030, 1037),
                                     (5000, 3, 2064, 2064), (6000, 3, 2064, 2064), (6000, 7, 2050, 2100),
                                     (5200, 4, 4208, 272)])
def test_rows_do_not_depend_on_their_neighbours(M, E, n, k, dx, out):
    say(f"neighbours M={M} E={E} n={n} k={k} dx={dx} {out}")
    x, xs = _quantized((M, n if dx else k), 1, "e4m3")
    w, ws = _quantized((E, n, k), 2, "e4m3", True)
    off = ints(_ragged(M, E, M))
    call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
    y = call(x, xs, w, ws, off, DT[out])
    r = np.random.default_rng(3)
    changed = np.sort(r.choice(M, M // 3, replace=False))
    rest = torch.from_numpy(np.setdiff1d(np.arange(M), changed)).cuda()
    changed = torch.from_numpy(changed).cuda()
    b = x.view(torch.uint8)
    b[changed] = torch.from_numpy(r.integers(0, 256, size=(len(changed), x.shape[1]), dtype=np.uint8)).cuda()
    b[changed[0::4]] = 0x7f
    for i, s in enumerate((float("nan"), float("inf"), 3e38, 0.0)):
        xs[changed[i::5]] = s
    z = call(x, xs, w, ws, off, DT[out])
    assert torch.equal(z[rest], y[rest]) and not torch.equal(z[changed], y[changed])


# ---------------------------------------------------------------- the norm's weight gradient
def _whole_rows(T, d, dtype, seed, live=None):
    """dy and h of whole numbers (zeros outside the live rows) and rstd of powers of two, with sum dy h rstd."""
    r = np.random.default_rng(seed)
    live = np.arange(T) if live is None else live
    a, b = (r.integers(-3, 4, size=(len(live), d)) for _ in range(2))
    rs = np.exp2(r.integers(-1, 2, size=len(live)))
    at = torch.from_numpy(live).cuda()
    dy, h = (torch.zeros((T, d), dtype=DT[dtype], device="cuda") for _ in range(2))
    rstd = torch.ones(T, device="cuda")
    dy[at], h[at], rstd[at] = dev(a, dtype), dev(b, dtype), dev(rs)
    want = (a * b * rs[:, None]).sum(0)
    assert (np.abs(a * b) * rs[:, None]).sum(0).max() * 2 < 2 ** 24
    return dy, h, rstd, want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", [(1, 1), (1, 2048), (5, 64), (33, 1024), (9, 1283), (700, 72), (2051, 130), (9000, 16),
                                 (16384, 64), (3, 5001), (4097, 513), (1000, 8192), (3001, 2050), (63, 20000),
                                 (64, 16400), (65, 20001), (515, 16392), (66000, 24)])
def test_weight_gradient_of_whole_numbers(T, d, dtype):
    say(f"dweight of whole numbers T={T} d={d} {dtype}")
    dy, h, rstd, want = _whole_rows(T, d, dtype, T + d)
    for w in (None, torch.full((d,), 0.5, dtype=DT[dtype], device="cuda")):      # w reaches dx only
        _, dw = mx.rms_norm_backward(dy, h, w, rstd)
        assert np.array_equal(host(dw), want)


@pytest.mark.parametrize("T,d,every", [((1 << 20) + 77, 2056, 997), (66000, 16400, 131), (1 << 24, 128, 8191)])
def test_weight_gradient_of_rows_past_4_gib(T, d, every):
    """Rows all over tensors past 4 GiB (2^31 elements and more), the last one among them."""
    assert T * d * 2 >= 2 ** 31
    say(f"dweight past 4 GiB T={T} d={d}")
    live = np.unique(np.append(np.arange(3, T, every), [0, T - 2, T - 1]))
    dy, h, rstd, want = _whole_rows(T, d, "bf16", T + d, live)
    _, dw = mx.rms_norm_backward(dy, h, None, rstd)
    assert np.array_equal(host(dw), want)
