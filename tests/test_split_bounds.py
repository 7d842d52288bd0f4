"""The arithmetic behind the float32 products on float16 and bfloat16 matrix instructions: what a
value's parts hold and what the products left out amount to, evaluated on the CPU (the bounds that
csrc/tile_gemm.h states and the GPU tests' tolerances count)."""
import numpy as np
import torch


def _values():
    """Significands around every border of the parts, and random ones, all of float32's bits."""
    r = np.random.default_rng(0)
    m = [1 + r.integers(0, 2 ** 23, 400_000) * 2.0 ** -23]
    for p in range(1, 24):
        for q in range(p, 24):
            m.append(np.array([1 + 2.0 ** -p + 2.0 ** -q - 2.0 ** -23, 1 + 2.0 ** -p, 2 - 2.0 ** -p - 2.0 ** -23 * (q > 12)]))
    v = np.concatenate(m)
    v = v[v < 2]
    return np.concatenate([v, -v]).astype(np.float32)


def _bf16(v):
    return torch.from_numpy(v).to(torch.bfloat16).to(torch.float32).numpy()


def test_two_float16_parts():
    v = _values() * np.float32(2.0 ** 13)
    hi = v.astype(np.float16).astype(np.float32)
    lo = (v - hi).astype(np.float16).astype(np.float32)
    v, hi, lo = (t.astype(np.float64) for t in (v, hi, lo))
    rest, part = np.abs((v - hi - lo) / v), np.abs(lo / v)
    assert 2.0 ** -23.01 < rest.max() <= 2.0 ** -23
    assert 2.0 ** -11.01 < part.max() <= 2.0 ** -11
    # lo lo' of two values: at most the square, 2^-22; root mean square over random ones 2^-24.5
    assert 2.0 ** -24.6 < np.mean(part[:400_000] ** 2) < 2.0 ** -24.4
    # values far below their row's largest (2^13): to 2^-38 of that
    small = (_values()[:, None] * 2.0 ** np.arange(-60, 12)).astype(np.float32)
    hi = small.astype(np.float16).astype(np.float32)
    lo = (small - hi).astype(np.float16)
    rest = np.abs(small.astype(np.float64) - hi - lo.astype(np.float64))
    assert (rest <= np.maximum(2.0 ** -23 * np.abs(small), 2.0 ** -25)).all()


def test_three_bfloat16_parts():
    v = _values()
    lift = np.float32(2.0 ** 24)
    for p in (-126, -60, 0, 60, 102):
        s = v * np.float32(2.0 ** p) * lift
        hi = _bf16(s)
        mid = _bf16(s - hi)
        lo = _bf16(s - hi - mid)
        s, hi, mid, lo = (t.astype(np.float64) for t in (s, hi, mid, lo))
        assert (hi + mid + lo == s).all()
        a, b = np.abs(mid / s).max(), np.abs(lo / s).max()
        assert a <= 2.0 ** -8 and b <= 2.0 ** -16
        assert 2 * a * b + b * b <= 2.0 ** -22.99       # mid lo' + lo mid' + lo lo'
    # subnormal values too
    tiny = (np.arange(1, 1 << 20, 7, dtype=np.float64) * 2.0 ** -149).astype(np.float32)
    s = tiny * lift
    hi = _bf16(s)
    mid = _bf16(s - hi)
    lo = _bf16(s - hi - mid)
    assert (hi.astype(np.float64) + mid + lo == tiny.astype(np.float64) * 2.0 ** 24).all()
