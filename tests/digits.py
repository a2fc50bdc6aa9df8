"""Activations as sums of E2M1 digits, restated in binary64, and the documented bounds of the
products that use them (include/mxfp4.h): a value enters to within 2^-22 of the largest of its
block (32 elements for MXFP4, 16 for NVFP4; NVFP4 also 2^-39 of the token's largest)."""
import numpy as np

import block_scaled_fp4_bf16_gb300 as mx

MX, NV = mx.MX_FMT_MXFP4, mx.MX_FMT_NVFP4
DIGITS = 8
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def block(fmt):
    return 32 if fmt == MX else 16


def e2m1(v):
    """The nearest E2M1 number, ties to the even code."""
    a = np.abs(v)[..., None]
    d = np.abs(a - GRID)
    best = d.min(-1, keepdims=True)
    code = np.where(d == best, np.arange(8) % 2 * 8 + np.arange(8), 99).argmin(-1)
    return np.sign(v) * GRID[code]


def shift(p):
    return 0 if p == 0 else 3 * p - 1


def exponent(top):
    """The least e with top <= 6 * 2^e (top > 0)."""
    m, e = np.frexp(np.where(top > 0, top, 1.0))  # top = m 2^e, m in [1/2, 1)
    return np.where(m > 0.75, e - 2, e - 3)


def as_digits(x, fmt, digits=DIGITS):
    """What `digits` E2M1 digits hold of x [rows, k]."""
    rows, k = x.shape
    b = x.reshape(rows, -1, block(fmt))
    e = exponent(np.abs(b).max(2, keepdims=True))
    if fmt == NV:
        row = np.maximum(exponent(np.abs(x).max(1)) - 8, -118)[:, None, None]
        e = row + np.clip(e - row, -9, 8)
    left, out = b * 2.0 ** -e, np.zeros_like(b)
    for p in range(digits):
        q = e2m1(left * 2.0 ** shift(p))
        out += q * 2.0 ** -shift(p)
        left = left - q * 2.0 ** -shift(p)
    return (out * 2.0 ** e).reshape(rows, k)


def loss(x, w, fmt):
    """The documented bound on what the digits of x [t, k] may change of x w^T: [t, rows]."""
    a, v, n = np.abs(x), np.abs(w), block(fmt)
    tol = 2.0 ** -22 * (a.reshape(len(a), -1, n).max(2) @ v.reshape(len(v), -1, n).sum(2).T)
    return tol if fmt == MX else tol + 2.0 ** -39 * a.max(1)[:, None] * v.sum(1)[None]


def ulp(v):
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))) - 7)


def silu(v):
    return v / (1.0 + np.exp(-v))


def expert(x, gate, up, down, fmt, act=silu):
    """D (act(G x) * U x) of rows x and its tolerance before the slots' sum: sums 1e-5 of the
    absolute ones (the GEMM tests' bound), the digits of x and of h by the documented bound,
    act's slope below 1.13, h's own roundings 2^-20."""
    g, u = x @ gate.T, x @ up.T
    eg = 1e-5 * (np.abs(x) @ np.abs(gate).T) + loss(x, gate, fmt)
    eu = 1e-5 * (np.abs(x) @ np.abs(up).T) + loss(x, up, fmt)
    h = act(g) * u
    dh = 1.13 * eg * np.abs(u) + np.abs(act(g)) * eu + eg * eu + 2.0 ** -20 * np.abs(h)
    tol = (dh + 1e-5 * np.abs(h)) @ np.abs(down).T + loss(np.abs(h) + dh, down, fmt)
    return h @ down.T, tol


class LowDigits:
    """An expert [n, 64] and rows x whose products are made of what lies 2^-12 to 2^-18 below
    the largest of a block: the largest have weights of zero.

    Columns 0..31 of x: per 16 one of 2^16 or so and small ones, each the whole of an up
    row's sum (code 1).  Column 32: 32, the gate of every row.  h then has the small ones of
    x, and per 16 one large one; a row of the down matrix takes one of the small ones."""

    def __init__(self, tokens, seed):
        rng = np.random.default_rng(seed)
        n = 32
        self.n, self.k = n, 64
        small = np.exp2(-rng.integers(0, 7, (tokens, n))) * (1 + rng.integers(0, 128, (tokens, n)) / 128.0)
        small *= rng.choice([-1.0, 1.0], (tokens, n))
        x = np.zeros((tokens, 64))
        x[:, :n] = small
        x[:, [0, 16]] = 2.0 ** 13 * 1.75
        x[:, 32] = 32.0
        self.x = x
        self.gate, self.up = np.zeros((n, 64)), np.zeros((n, 64))
        self.gate[:, 32] = 1.0
        self.few = [i for i in range(n) if i % 16]
        self.up[np.arange(n), np.arange(n)] = 1.0
        self.down = np.zeros((64, n))
        self.down[np.arange(64), rng.choice(self.few, 64)] = rng.choice([-1.0, 1.0, 1.5, 3.0], 64)


def unpacked_tensors(values, fmt):
    """(packed codes, scale bytes [rows, blocks]) of E2M1 values under scales of 1."""
    code = np.searchsorted(GRID, np.abs(values)) + np.where(values < 0, 8, 0)
    assert (GRID[code & 7] == np.abs(values)).all()
    packed = (code[:, ::2] | code[:, 1::2] << 4).astype(np.uint8)
    return packed, np.full((len(values), values.shape[1] // block(fmt)), 127 if fmt == MX else 0x38, np.uint8)
