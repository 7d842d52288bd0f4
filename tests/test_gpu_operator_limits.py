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
