"""Rotation at positions over the whole range of 64 bits: the angle is the exact product's."""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PI = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
POSITIONS = [2 ** 62 + 12345, -2 ** 62 - 99999, 2 ** 63 - 1, -2 ** 63, 2 ** 55 + 7, -2 ** 48 - 1, 1, -1]


@pytest.mark.parametrize("D", [64, 62])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_the_farthest_positions(lib, D, sign, interleaved):
    """Tolerance as in test_gpu_append: half a step, and 24 2^-24 of a pair's features."""
    T, half = len(POSITIONS), D // 2
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn(T, 3, D, generator=g, device="cuda").half()
    cache = torch.zeros(1, 16, 1, D, dtype=torch.float16, device="cuda")
    freq = sign * torch.tensor([1e4 ** (-2 * i / D) for i in range(half)], device="cuda")
    freq[1], freq[2], freq[3] = 3.75 * sign, 2.0 ** -140, 1000.5
    out = lib.rope_append(rows[:, :1], rows[:, 1:2], rows[:, 2:], cache, cache.clone(), torch.full((T,), -1, device="cuda"),
                          torch.tensor(POSITIONS, device="cuda"), freq, interleaved=interleaved)
    assert lib.get_last_error() == 0
    x, got = rows[:, 0].double().cpu().numpy(), out[:, 0].double().cpu().numpy()
    a, b = (slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, half), slice(half, D))
    for t, p in enumerate(POSITIONS):
        w = np.array([float(Fraction(p) * Fraction(float(f)) % (2 * PI)) for f in freq.cpu()])
        size = np.abs(x[t, a]) + np.abs(x[t, b])
        for at, want in ((a, x[t, a] * np.cos(w) - x[t, b] * np.sin(w)), (b, x[t, b] * np.cos(w) + x[t, a] * np.sin(w))):
            assert (np.abs(got[t, at] - want) <= 2.0 ** -11 * np.abs(want) * 1.001 + 24 * 2.0 ** -24 * size + 2.0 ** -25).all(), (p, got[t, at] - want)
