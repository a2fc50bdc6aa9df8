"""mx_linear_bf16 at the ends of binary32's range: block scales near 2^127 under small
activations, activations near the type's largest under a small tensor scale.  The formula's
result is finite, though a sum in other units on the way to it need not be.

Tolerances: those of the other few-token tests (1e-5 sum |x||w|, and what the activations'
form may lose), from the formula in binary64.
"""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
import oracle
from block_scaled_fp4_bf16_gb300 import synth
from tests.gpu_helpers import bf16_bits_to_f64
from tests.test_gpu_few_tokens import (FMTS, MX, NV, Weight, assert_close, linear_ref, run_linear, ulp,
                                       x_bits)
from tests.test_gpu_linear_workspace import Wide, pick, reference, run

pytestmark = pytest.mark.gpu

# every instance of the kernel without a workspace: rows of an item, tokens of a product
DIRECT = [(3, 96, 1056), (8, 9760, 160), (13, 160, 1056), (16, 9760, 160), (32, 160, 544), (1, 64, 8192)]
BIG = 0x7F7F  # the largest BF16 number


def scaled(bits, exponents):
    x = bf16_bits_to_f64(bits) * 2.0 ** np.asarray(exponents, dtype=np.float64)[:, None]
    return synth.f32_to_bf16_bits(x.astype(np.float32))


@pytest.mark.parametrize("lo,hi", [(232, 254), (110, 254)])
@pytest.mark.parametrize("tokens,n,k", DIRECT)
def test_large_block_scales(tokens, n, k, lo, hi):
    w = Weight(n, k, MX, 401, lo, hi)
    bits = scaled(x_bits(tokens, k, 402), [(-20, -60, -100)[t % 3] for t in range(tokens)])
    ref, tol = linear_ref(bits, w)
    assert np.abs(ref).max() < 1e38
    assert_close(run_linear(bits, w), ref, tol, "fp32")
    assert_close(run_linear(bits, w, out_fp32=False), ref, tol + ulp(ref), "bf16")


def test_one_large_scale_among_ordinary_ones():
    """x about 1, codes 6, a scale of 2^107: 2^114 of sum."""
    n, k = 64, 256
    w = Weight(n, k, MX, 411, 127, 127)
    w.codes[:] = 0x77
    w.value = np.full((n, k), 6.0)
    bits = synth.f32_to_bf16_bits(np.ones((2, k), np.float32))
    s = np.full((n, k // 32), 127, np.uint8)
    s[7, 3] = 107 + 127
    w.value[7, 96:128] *= 2.0 ** 107
    w.scales = oracle.scale_tile(s)
    ref, tol = linear_ref(bits, w)
    assert_close(run_linear(bits, w), ref, tol, "one block")


@pytest.mark.parametrize("tokens,n,k", DIRECT)
def test_large_activations_under_a_small_tensor_scale(tokens, n, k):
    """A token of the type's largest magnitudes; the others' bits do not change for it."""
    w = Weight(n, k, NV, 421, 0x20, 0x7E)
    w.value *= 2.0 ** -30 / float(w.ts)
    w.ts = np.float32(2.0 ** -30)
    bits = x_bits(tokens, k, 422)
    clean = run_linear(bits, w)
    bits[0] = BIG | (bits[0] & 0x8000)
    ref, tol = linear_ref(bits, w)
    got = run_linear(bits, w)
    assert np.abs(ref).max() < 1e38
    assert_close(got, ref, tol, "largest")
    assert (got[1:] == clean[1:]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_results_beyond_the_range_stay_infinite(fmt):
    """All products of one sign: the formula's own result is past binary32."""
    w = Weight(96, 416, fmt, 431, *((200, 200) if fmt == MX else (0x7E, 0x7E)))
    w.codes &= 0x77  # no negative code
    if fmt == NV:
        w.ts = np.float32(2.0 ** 40)
    bits = np.full((2, 416), BIG, np.uint16)
    bits[1] = BIG | 0x8000
    got = run_linear(bits, w)
    assert (got[0] == np.inf).all() and (got[1] == -np.inf).all()


# with a workspace: one, two, four and eight columns of digits' blocks; two and more CTAs a tile
WIDE = [(4, 2464, 28768), (8, 8224, 8224), (16, 12320, 4128), (20, 8224, 8224)]


@pytest.mark.parametrize("tokens,n,k", WIDE)
def test_large_block_scales_with_a_workspace(tokens, n, k):
    assert mx.mx_linear_workspace_bytes(tokens, k, n, MX) > 0
    w = Wide(n, k, MX, 441, 110, 254)
    bits = scaled(x_bits(tokens, k, 442), [(-20, -60, -100)[t % 3] for t in range(tokens)])
    ref, tol = reference(bits, w)
    assert np.abs(ref).max() < 1e38
    assert_close(pick(run(bits, w), w), ref, tol, "fp32")


@pytest.mark.parametrize("tokens,n,k", WIDE)
def test_large_activations_under_a_small_tensor_scale_with_a_workspace(tokens, n, k):
    assert mx.mx_linear_workspace_bytes(tokens, k, n, NV) > 0
    w, bits = Wide(n, k, NV, 451, 0x20, 0x7E), x_bits(tokens, k, 452)
    w.ts.fill_(2.0 ** -30)
    clean = run(bits, w)
    bits[0] = BIG | (bits[0] & 0x8000)
    ref, tol = reference(bits, w)
    assert np.abs(ref).max() < 1e38
    got = run(bits, w)
    assert_close(pick(got, w), ref, tol, "largest")
    assert torch.equal(got[1:], clean[1:])
    assert_close(pick(run(bits, w, out_fp32=False), w), ref, tol + ulp(ref), "bf16")


@pytest.mark.parametrize("fmt", FMTS)
def test_infinities_with_a_workspace_whose_weights_are_next_to_nothing(fmt):
    """inf times the least weight other than zero is inf, and times zero NaN."""
    t, n, k = 3, 8224, 8224
    w, bits = Wide(n, k, fmt, 461, *((0, 0) if fmt == MX else (1, 1))), x_bits(t, k, 462)
    if fmt == NV:
        w.ts.fill_(2.0 ** -140)
    bits[1, 100] = 0x7F80
    got, v = pick(run(bits, w), w), w.value()
    zero = v[:, 100] == 0
    assert np.isnan(got[1][zero]).all() and (got[1][~zero] == np.sign(v[~zero, 100]) * np.inf).all()
    assert np.isfinite(got[[0, 2]]).all()
