"""The weights of mx_sample: the kernel's binary32 operations, one by one (numpy), against the
exponential to 60 digits.  They are IEEE operations, so the kernel's results are these."""
import os
import re
from decimal import Decimal, getcontext

import numpy as np

from block_scaled_fp4_bf16_gb300 import build as _build

getcontext().prec = 60
f = np.float32


def source():
    with open(os.path.join(_build.CSRC, "sample.cu")) as fh:
        return fh.read()


def fma(a, b, c):
    """One rounding: a b is exact in binary64, and its sum with c is off by 2^-53 before the last."""
    return f(np.float64(a) * np.float64(b) + np.float64(c))


def bits(x):
    return int(np.asarray(x, f).view(np.uint32))


def roots():
    return [int(v, 16) for v in re.search(r"kRoot\[8\] = \{([^}]*)\}", source()).group(1).replace("ull", "").split(",")]


def table():
    out = []
    for j in range(256):
        v = 1 << 63
        for i, r in enumerate(roots()):
            if j >> (7 - i) & 1:
                p = v * r
                v = (p >> 64 << 1 | p >> 63 & 1) & (2 ** 64 - 1)
        out.append((f(v >> 40) * f(2.0 ** -23), f(f(v & (1 << 40) - 1) * f(2.0 ** -63))))
    return out


TABLE = table()


def weight(l, top, temperature):
    c = [f(float.fromhex(v)) for v in ("0x1.715476p+0", "0x1.4ae0cp-26")]
    t = min(max(f(temperature), f(2.0 ** -100)), f(2.0 ** 100))
    hi = f(c[0] / t)
    lo = f(f(fma(-hi, t, c[0]) + c[1]) / t)
    nt = f(-top)
    d = f(l + nt)
    b = f(d - l)
    e = f(f(l - f(d - b)) + f(nt - b))
    p = f(d * f(-hi))
    if not p < 46:
        return 0
    pe = fma(d, lo, fma(e, hi, fma(d, hi, p)))
    magic = f(1.5 * 2 ** 23)
    kb = fma(p, f(-256), magic)
    r = fma(f(kb - magic), f(2.0 ** -8), p)
    ln2, low = f(float.fromhex("0x1.62e43p-1")), f(float.fromhex("-0x1.05c61p-29"))
    yh, ny = f(r * -ln2), f(r * ln2)
    yl = fma(pe, ln2, fma(r, -low, fma(r, -ln2, ny)))
    c2 = fma(ny, fma(ny, f(1 / 24), f(-1 / 6)), f(0.5))
    ql = fma(yl, yh, fma(f(ny * ny), c2, yl))
    qh = f(yh + ql)
    qe = f(ql - f(qh - yh))
    th, tl = TABLE[bits(kb) & 255]
    m = f(th * qh)
    me = fma(th, qh, f(-m))
    s = f(th + m)
    sl = f(f(m - f(s - th)) + f(fma(th, qe, fma(tl, qh, tl)) + me))
    scale = np.uint32(((bits(kb) >> 8 << 23) + 0x3F800000) & 0xFFFFFFFF).view(f)
    v, vl = f(s * scale), f(sl * scale)
    high = f(v + f(4))
    low = f(f(f(v - f(high - f(4))) + vl) + f(1.5 * 2 ** -20))
    return ((bits(high) - 0x40800000) << 22) + bits(low) - 0x35C00000


def test_the_table_is_of_powers_of_two():
    for j, (h, l) in enumerate(TABLE):
        want = Decimal(2) ** (Decimal(j) / 256)
        assert abs(Decimal(float(h)) + Decimal(float(l)) - want) < Decimal(2) ** -45


def test_weights_are_within_their_stated_error():
    rng = np.random.default_rng(0)
    for _ in range(6000):
        top, t = f(rng.normal() * 10), f(np.exp(rng.normal() * 2))
        l = f(float(top) - abs(rng.normal()) * rng.choice([1e-6, 0.01, 1, 10, 25]) * float(t))
        got = weight(l, top, t)
        want = ((Decimal(float(l)) - Decimal(float(top))) / Decimal(float(t))).exp()
        # two roundings to units of 2^-43 (half a unit each) and 2^-40 relative
        assert abs(Decimal(got) / 2 ** 43 - want) <= Decimal(2) ** -43 + want * Decimal(2) ** -40
        assert got >= 0
    assert weight(f(1.5), f(1.5), f(0.7)) == 1 << 43
    assert weight(f(-1e30), f(3e38), f(1.0)) == 0 and weight(f(0.0), f(50.0), f(1.0)) == 0


def test_the_kernel_has_these_constants():
    text = source()
    for v in ("0x1.715476p+0f", "0x1.4ae0cp-26f", "0x1.8p23f", "0x1.62e43p-1f", "-0x1.05c61p-29f", "1.0f / 24.0f", "-1.0f / 6.0f",
              "0x1.8p-20f", "0x40800000u", "0x35C00000u", "0x3F800000u"):
        assert v in text, v
