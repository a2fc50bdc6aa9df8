"""The angles of mx_qk_norm_rope_bf16 at large frequencies and far positions, against integers of 300
bits.  Positions are chosen so that the angle is all but a whole number of turns: the sine is then small, and its
BF16 output shows the angle itself.

The phase is right to 2^-32 of a turn; a phase below 2^-20 of a turn has 13 bits of its 32 and is
exact in binary32.  So the sine of phi (2 pi 2^-20 at most) is off by 2 pi 2^-32, by the sine's 2^-22 and by
half a BF16 step of itself, 2^-8."""
import math

import numpy as np
import pytest
import torch
from decimal import Decimal, getcontext

import block_scaled_fp4_bf16_gb300 as mx

pytestmark = pytest.mark.gpu

BITS = 300


def two_pi_inverse():
    """floor(2^BITS / 2 pi), from pi = 16 atan(1/5) - 4 atan(1/239) (Machin)."""
    getcontext().prec = 120

    def atan(n):
        x = Decimal(1) / n
        term, s, k = x, x, 1
        while abs(term) > Decimal(10) ** -115:
            term = -term / (n * n)
            k += 2
            s += term / k
        return s
    return int((Decimal(2) ** BITS / (2 * (16 * atan(5) - 4 * atan(239)))).to_integral_value())


INVERSE = two_pi_inverse()


def phase(f, position):
    """The angle in turns, in -1/2 .. 1/2."""
    m, e = math.frexp(f)
    p = (int(m * 2 ** 24) * INVERSE * position << max(e - 24, 0)) >> max(24 - e, 0)
    p &= (1 << BITS) - 1
    return (p - (1 << BITS) if p >> (BITS - 1) else p) / 2.0 ** BITS


FREQUENCIES = [65536.0, 65535.996, -60000.5, 30011.25, 4097.0, 1000.5, -17.25, 16.0, 3.1415927, 1.0, 0.70710677, 2.0 ** -10]


def near_whole_turns(f, low, high, wanted, rng):
    """Positions for which |phase| < 2^-20, and is not all but 0 either."""
    found = []
    while len(found) < wanted:
        t = int(abs(phase(f, 1)) * 2.0 ** 64 if phase(f, 1) >= 0 else (1 + phase(f, 1)) * 2.0 ** 64)
        start = int(rng.integers(low, high - 2 ** 21))
        p = np.arange(start, start + 2 ** 21, dtype=np.uint64)
        q = (p * np.uint64(t)).view(np.int64)  # (a first look: off by as much as the constant's 64 bits are)
        for at in p[np.abs(q) < 2 ** 46].tolist():
            x = phase(f, at)
            if 2.0 ** -24 < abs(x) < 2.0 ** -20:
                found.append(at)
    return found[:wanted]


@pytest.mark.parametrize("interleaved", [False, True])
def test_small_angles_at_far_positions(interleaved):
    rng = np.random.default_rng(0)
    dim, n = 32, 16
    for f in (float(np.float32(f)) for f in FREQUENCIES):
        positions = near_whole_turns(f, 2 ** 30, 2 ** 31 - 1, 6, rng)
        positions += [-p for p in positions]
        inv = torch.full((n,), f, dtype=torch.float32, device="cuda")
        norm = mx.qk_norm(1, 0, dim, None, None, inv, dim, interleaved)
        x = torch.zeros(len(positions), dim, dtype=torch.bfloat16, device="cuda")
        first = slice(0, None, 2) if interleaved else slice(0, n)
        second = slice(1, None, 2) if interleaved else slice(n, None)
        x[:, first] = 1.0
        pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
        y = torch.empty_like(x)
        mx.mx_qk_norm_rope_bf16(x, dim, None, 0, len(positions), pos, norm, y, dim, None, 0)
        got = y.double().cpu().numpy()
        for i, p in enumerate(positions):
            want = math.sin(2 * math.pi * phase(f, p))
            assert (got[i, first] == 1.0).all()
            bound = 2 * math.pi * 2.0 ** -32 + (2.0 ** -8 + 2.0 ** -22) * abs(want)
            assert (np.abs(got[i, second] - want) <= bound).all(), (f, p, want, got[i, second][0])
        # the gradients turn back by the same angles
        g = torch.empty_like(x)
        mx.mx_qk_norm_rope_backward_bf16(x, dim, None, 0, x, dim, None, 0, len(positions), pos, norm, g, dim, None, 0)
        assert torch.equal(g[:, second], -y[:, second]) and torch.equal(g[:, first], y[:, first])
    assert mx.mx_device_status() == 0
