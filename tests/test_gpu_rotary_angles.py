"""Angles of the rotated append for large and negative frequencies at the furthest positions, against angles from
whole-number arithmetic: a product in FP64 is off by whole turns there."""

from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_conv_rotary import DEV, HALF, TINY, Rotary, f64  # noqa: E402
from tests.test_gpu_delta_batch import vq3  # noqa: E402,F401

pytestmark = pytest.mark.gpu
PI = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10**62)


def turned(x, positions, freq):
    half = len(freq)
    turns = [[Fraction(float(f)) * p / (2 * PI) for f in freq] for p in positions]
    angle = 2 * np.pi * np.array([[float(t - round(t)) for t in row] for row in turns])[:, None]
    a, b = x[..., :half], x[..., half : 2 * half]
    c, s = np.cos(angle), np.sin(angle)
    return np.concatenate([a * c - b * s, b * c + a * s], -1), np.concatenate([np.hypot(a, b)] * 2, -1)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_frequencies(vq3, dtype):  # noqa: F811
    c = Rotary(8, [2**31 - 1, 2**30 + 1, 10**9 + 7, 16777217, 2**31 - 2, 1, 0], dim=64, rotated=64, dtype=dtype)
    c.freq[:16] = torch.tensor([100.5, 1000.3, -7777.7, 3e4, 1e6, -1e6, 12345678.0, 1e9, -1e-12, -1e-17, -1.0, -0.3, 2.0**30,
                                -(2.0**-40), 6.2831855, 3.1415927])
    got = c.run(vq3)
    # a turn of 2^-25 (2^-22.3 radians), products and sums in FP32: within 2^-21 of the pair's length
    for out, x in ((got, c.q), (torch.stack([c.pages[0][s // 16, s % 16] for s in c.slots]), c.k)):
        ref, size = turned(f64(x), c.positions, c.freq.numpy())
        assert (np.abs(f64(out) - ref) <= HALF[dtype] * np.abs(ref) + (1 + HALF[dtype]) * 2.0**-21 * size + TINY[dtype]).all()
