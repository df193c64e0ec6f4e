"""Rotary positions (cp_rope) at angles whose sine or cosine is small."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import context_zigzag_cp_b200 as cz
from helpers import f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "adjacent"])
def test_small_angles_keep_their_digits(layout):
    """Pairs (1, 0) and (0, 1) turned by angles near 0 and near the quarter turns: sine and cosine relative to
    themselves.  Half a bf16 step, and the fp32 steps before it (the angle's 2^-24, sine and cosine to 2 of 2^-23, one product)."""
    D, N = 64, 48
    near = np.concatenate([[0, 0, 0, 0], np.repeat([1, 2, 3, 4, 5], 5), [0, 0, 0]])
    tiny = np.array([2.5e-6, 1e-7, -3e-5, 7.7e-9] + [1e-5, -1e-6, 3e-8, 2e-4, -7e-3] * 5 + [1e-4, -2e-10, 5e-3])
    f = near * (np.pi / 2) + tiny
    assert len(f) == D // 2
    pos = np.zeros((1, N), np.int32)
    pos[0] = np.arange(N)
    x = torch.zeros(1, 2, N, D)
    first, second = (slice(0, 32), slice(32, 64)) if layout == "half" else (slice(0, 64, 2), slice(1, 64, 2))
    x[0, 0, :, first], x[0, 1, :, second] = 1, 1
    for inverse in (False, True):
        y = f64(cz.rope([x.bfloat16().cuda()], torch.from_numpy(f).cuda(), positions=torch.from_numpy(pos).cuda(),
                        layout=layout, inverse=inverse)[0])[0]
        # the angle is that of the 64-bit frequency: its own last place is 2^-53 of it, the quarter turns' remainders are
        # taken from pi to 32 digits
        half_pi = Fraction(31415926535897932384626433832795, 2 * 10 ** 31)
        c, s = np.zeros((N, 32)), np.zeros((N, 32))
        for n in range(N):
            for i in range(32):
                a = Fraction(float(f[i])) * n
                turns = round(a / half_pi)
                r = float(a - turns * half_pi)
                cs, sn = math.cos(r), math.sin(r)
                for _ in range(turns % 4):
                    cs, sn = -sn, cs
                c[n, i], s[n, i] = cs, sn
        s = -s if inverse else s
        for got, want in ((y[0][:, first], c), (y[0][:, second], s), (y[1][:, first], -s), (y[1][:, second], c)):
            # two units in the last place of sine and cosine, the angle's and the product's roundings
            assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -20) + 2.0 ** -64 * 2 * np.pi * N).all()
