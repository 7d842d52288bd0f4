"""Operators at the largest numbers of rows that they accept, where counts of threads, tiles and
rows come near 2^31 and 2^32.  Inputs are chosen so that every result is exact, or stands in
a few rows that a small call gives as well."""
import numpy as np
import pytest
import torch

from parity_helpers import say
from test_gpu_quantized import _routing, dev, ints

pytestmark = pytest.mark.gpu

mx = pytest.importorskip("mixture_experts_ffn_fp32_amd")


def test_balance_loss_of_more_chunks_than_one_launch_has_blocks():
    """T / 64 chunks of 512 threads are 2^32 threads and more.  Scores are powers of two, so the
    sums are exact; the last sequence is as that of a small call."""
    T, N, tail = (1 << 29) + 1000, 3, 1000
    say(f"balance loss T={T}")
    s, idx = _routing(tail, N, 1, 3)
    scores = torch.tensor([0.5, 0.25, 0.125], device="cuda").expand(T, N).contiguous()
    scores[-tail:] = dev(s)
    at = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    at[1::2] = 1
    at[-tail:] = torch.from_numpy(idx).cuda()
    cuts = [0, (1 << 28) + 6, T - tail, T]
    b = mx.balance_loss(scores, at, ints(cuts))
    c = mx.balance_loss(dev(s), torch.from_numpy(idx).cuda())
    for q in range(2):
        n = cuts[q + 1] - cuts[q]                   # even, and starts at an even row
        assert b["counts"][q].tolist() == [n // 2, n // 2, 0]
        assert b["P"][q].tolist() == [0.5, 0.25, 0.125]
        # f = 3/2 of the experts 0 and 1: 3/2 (1/2 + 1/4)
        assert b["losses"][q, 0].item() == 1.125
    for name in ("counts", "P", "losses", "slopes"):
        assert torch.equal(b[name][2], c[name][0]), name
    z = mx.balance_loss_backward(scores, b["slopes"], None, ints(cuts))
    assert torch.equal(z[-tail:], mx.balance_loss_backward(dev(s), c["slopes"]))
    for q in range(2):
        at0, at1 = cuts[q], cuts[q + 1]
        assert (z[at0:at1] == z[at0]).all()
        slope = b["slopes"][q, 0].double()
        row = scores[at0].double()
        assert torch.allclose(z[at0].double(), row * (slope - row @ slope), rtol=0, atol=8 * 2.0 ** -24 *
                              float(slope.max()))


def _rows_of_the_most(M, k, dtype, seed):
    """M rows of k zeros whose last ones are whole numbers, and those."""
    tail = np.random.default_rng(seed).integers(-3, 4, size=(300, k))
    x = torch.zeros((M, k), dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device="cuda").view(dtype)
    last = torch.from_numpy(tail.astype(np.float32)).to(dtype).cuda()
    (x.view(torch.uint8) if dtype == torch.float8_e4m3fn else x)[-300:] = (
        last.view(torch.uint8) if dtype == torch.float8_e4m3fn else last)
    return x, tail


@pytest.mark.parametrize("dx", [False, True])
def test_eight_bit_product_of_the_most_rows(dx):
    """One group of 2^31 - 1 rows: its tiles are counted without an overflow."""
    M, n, k = 2147483647, 16, 16
    say(f"8-bit product of {M} rows dx={dx}")
    x, tail = _rows_of_the_most(M, 16, torch.float8_e4m3fn, 1)
    xs = torch.ones((M, 1), device="cuda")
    wv = np.random.default_rng(2).integers(-3, 4, size=(n, k))
    w = torch.from_numpy(wv[None].astype(np.float32)).to(torch.float8_e4m3fn).cuda()
    call = mx.grouped_matmul_quantized_dx if dx else mx.grouped_matmul_quantized
    out = torch.full((M, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    call(x, xs, w, torch.ones((1, 1, 1), device="cuda"), None, out=out)
    want = tail @ (wv if dx else wv.T)              # at most 144: exact in bfloat16
    assert np.array_equal(out[-300:].float().cpu().numpy(), want)
    for a in range(0, M - 300, 1 << 28):
        assert not out[a:min(a + (1 << 28), M - 300)].any(), a


def test_weight_gradient_of_the_most_rows():
    """The same of bfloat16 rows: a contraction of 2^31 - 1 indices (y and dx of so many rows need
    more memory than there is)."""
    M, n = 2147483647, 8
    say(f"weight gradient of {M} rows")
    x, tail = _rows_of_the_most(M, n, torch.bfloat16, 3)
    w = torch.zeros((1, n, n), dtype=torch.bfloat16, device="cuda")
    _, dw = mx.grouped_matmul_backward(x, w, ints([0, M]), x, need_dx=False)
    assert np.array_equal(dw[0].cpu().numpy(), tail.T @ tail)      # at most 2700: exact


def test_balance_loss_of_the_most_rows():
    T = 2147483647
    say(f"balance loss T={T}")
    s = torch.ones((T, 1), device="cuda")
    idx = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    b = mx.balance_loss(s, idx)
    assert b["counts"].item() == T and b["P"].item() == 1 and b["losses"][0].tolist() == [1, 0]
    assert b["slopes"][0, 0].item() == np.float32(1 / T)
    z = mx.balance_loss_backward(s, b["slopes"])
    for a in range(0, T, 1 << 28):
        assert not z[a:a + (1 << 28)].any(), a              # s (c - s c) with s = 1
