"""Frequencies of any size, against 50 decimal digits: what an angle may be off by (gdn.h).

theta_j is formed in 64-bit floats: its power (the exponent's rounding counts |ln base^(-2j/rot)| times, the
function once), the division by factor, 2 pi and the division by it make less than 4 + |ln| roundings of 2^-53
of it.  Nothing is lost after that but the fraction's last place, 2^-65 of a turn a position.  Sine and
cosine are off by as many radians, and by 4 roundings of 2^-24 (as in the other tests of these calls:
sincospi, the correction and the scale)."""
from decimal import Decimal, getcontext
import math

import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi

pytestmark = pytest.mark.gpu
getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def turns(base, factor, rot):
    """theta_j / 2 pi exactly, and what 64-bit floats may be off by."""
    out, off = [], []
    for j in range(rot // 2):
        log = -2 * j / Decimal(rot) * Decimal(base).ln()
        t = log.exp() / Decimal(factor) / (2 * PI)
        out.append(t)
        off.append(float(t) * (4 + abs(float(log))) * 2.0 ** -53 + 2.0 ** -65)
    return out, off


@pytest.mark.parametrize("base,factor", [
    (10000.0, 1.0), (500000.0, 4.0), (0.5, 1.0), (1e-2, 1.0), (1e-4, 1.0), (10000.0, 1e-3), (1e-6, 0.01),
    (1e9, 0.25), (1.0, 0.7)])
def test_angles_are_off_by_what_is_stated(base, factor):
    d = 64
    positions = [0, 1, -1, 77, 4095, -100003, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31]
    x = torch.zeros(len(positions), 1, d, device="cuda")
    x[..., :d // 2] = 1.0  # a = 1, b = 0: cosine and sine
    rope = abi.Rope(d, base=base, factor=factor)
    y, _ = abi.gdn_rope(rope, torch.tensor(positions, dtype=torch.int32, device="cuda"), x,
                        q_out=torch.empty_like(x))
    y = y[:, 0].double().cpu().numpy()
    exact, off = turns(base, factor, d)
    for i, p in enumerate(positions):
        for j in range(d // 2):
            t = exact[j] * p
            angle = 2 * math.pi * float(t - t.to_integral_value())
            tol = 2 * math.pi * abs(p) * off[j] + 4 * 2.0 ** -24
            assert abs(y[i, j] - math.cos(angle)) <= tol, (p, j)
            assert abs(y[i, d // 2 + j] - math.sin(angle)) <= tol, (p, j)
    if base >= 1 and factor >= 1:  # the simple form of the bound
        assert max(off) <= 2.0 ** -52
