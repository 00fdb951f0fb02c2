"""Rotary positions whose frequencies are far above one radian per unit, at positions up to 2^31.  The reference
reduces the angle in whole numbers: pos * freq is a fraction, 2 pi is taken to 320 bits.

Bound: test_rope_gpu.py's 6e-7 (|x_a| + |x_b|) + 2^-8 |y|, and the step's own rounding, 2^-65 revolutions,
2^31 2^-65 2 pi = 4e-10, far inside what the 6e-7 leaves."""
from fractions import Fraction
from math import cos, sin

import numpy as np
import pytest
import torch

from tests.pi_bits import two_pi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("freqs", [[1.0, 0.3, 6.0, 100.0], [1e3, 1e4, 1e5, 3.7e6], [-1e9, 2.5e15, 1.7e19, -3e12]])
def test_far_positions_and_large_frequencies(freqs):
    import top_routed_block_b200 as fv
    pos = [2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 12345, 99991, 1, 0, -7]
    x = torch.from_numpy(np.random.default_rng(3).standard_normal((1, 2, len(pos), 64))).to(torch.bfloat16).cuda()
    rope = fv.RopeAxes(np.array(freqs), np.zeros(len(freqs), np.int32))
    y, _ = fv.fvattn_rope(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda")[:, None], rope)
    got, x = y.double().cpu().numpy(), x.double().cpu().numpy()
    for t, p in enumerate(pos):
        for j, f in enumerate(freqs):
            turns = p * Fraction(f) / two_pi(320)
            angle = float((turns - round(turns)) * two_pi(320))
            a, b = x[0, :, t, 2 * j], x[0, :, t, 2 * j + 1]
            for c, want in ((2 * j, a * cos(angle) - b * sin(angle)), (2 * j + 1, b * cos(angle) + a * sin(angle))):
                tol = 2.0 ** -8 * np.abs(want) + 6e-7 * (np.abs(a) + np.abs(b))
                assert (np.abs(got[0, :, t, c] - want) <= tol).all(), (p, f, got[0, :, t, c], want)
