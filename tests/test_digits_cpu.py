"""The digits of activations, restated: eight of them meet the documented bounds, and the
tolerances of the GPU tests that build on those bounds tell seven from eight."""
import numpy as np
import pytest

from tests import digits as d


def bf16(v):
    u = v.astype(np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("fmt", [d.MX, d.NV])
def test_eight_digits_meet_the_bound(fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 256)) * np.exp2(rng.integers(-18, 1, (40, 256)))
    x[1] = bf16(x[1])
    x[2, ::16] = [6.0] * 16
    x[3] = 0.0
    top = np.abs(x).reshape(40, -1, d.block(fmt)).max(2).repeat(d.block(fmt), 1)
    bound = 2.0 ** -22 * top + (0 if fmt == d.MX else 2.0 ** -39 * np.abs(x).max(1)[:, None])
    err = np.abs(d.as_digits(x, fmt) - x)
    assert (err <= bound).all()
    # and a BF16 value not below 2^-13 of its block's largest is exact
    b = bf16(x)
    top = np.abs(b).reshape(40, -1, d.block(fmt)).max(2).repeat(d.block(fmt), 1)
    far = np.abs(b) >= 2.0 ** -13 * top
    if fmt == d.NV:
        far &= top >= 2.0 ** -16 * np.abs(b).max(1)[:, None]
    assert far.sum() > 5000 and (d.as_digits(b, fmt) == b)[far].all()
    assert (np.abs(d.as_digits(x, fmt, 7) - x) > bound).any()


@pytest.mark.parametrize("fmt", [d.MX, d.NV])
@pytest.mark.parametrize("of", ["x", "h"])
def test_fewer_digits_would_be_seen(fmt, of):
    """The low-digit case of the experts' GPU test: with seven or fewer digits of x, or of h,
    outputs leave its tolerance; with eight none does."""
    c = d.LowDigits(6, 3)
    y, tol = d.expert(c.x, c.gate, c.up, c.down, fmt)
    for n in (8, 7, 6, 4):
        x = d.as_digits(c.x, fmt, n if of == "x" else 8)
        h = d.silu(x @ c.gate.T) * (x @ c.up.T)
        got = bf16(d.as_digits(h, fmt, n if of == "h" else 8) @ c.down.T)
        bad = np.abs(got - y) > tol + d.ulp(y)
        assert bad.any() == (n < 8), n


@pytest.mark.parametrize("fmt", [d.MX, d.NV])
def test_fewer_digits_of_a_linear_would_be_seen(fmt):
    rng = np.random.default_rng(5)
    x, w = low_linear(rng, 5, 512, 64, fmt)
    tol = 1e-5 * (np.abs(x) @ np.abs(w).T) + d.loss(x, w, fmt)
    for n in (8, 7, 6, 4):
        bad = np.abs(d.as_digits(x, fmt, n) @ w.T - x @ w.T) > tol
        assert bad.any() == (n < 8), n


def low_linear(rng, tokens, k, rows, fmt):
    """x [tokens, k] with one large element a block, whose weights are zero, and w [rows, k]
    that takes one of the others of one block."""
    n = d.block(fmt)
    x = rng.choice([-1.0, 1.0], (tokens, k)) * np.exp2(-rng.integers(0, 7, (tokens, k)))
    x *= 1 + rng.integers(0, 128, (tokens, k)) / 128.0
    x[:, ::n] = 2.0 ** 13 * 1.75
    w = np.zeros((rows, k))
    at = rng.integers(0, k // n, rows) * n + rng.integers(1, n, rows)
    w[np.arange(rows), at] = rng.choice([-1.0, 1.0, 1.5, 3.0], rows)
    return x, w
