"""The attention's weights where the output nearly cancels, so that their rounding shows and not the
output's own.

A row has five tokens that matter; queries and keys have one channel, so that a product is exact.
Bound relative to sum w |v| / sum w: an exponent in powers of two is off by three roundings of its
scaling (2^-24 of at most 4 each) and one of its sum with the lift (2^-20), the exponential by 2^-22:
2^-19 in all, and as much for the sum of weights; binary32 sums and the rescaling at up to seven
new maxima 2^-18; the weights themselves 2^-21.  Together less than 2^-16 (a weight in one FP16
number would be off by up to 2^-11, which comes to some 2^-13 here)."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests import decode_ref as ref
from tests.test_gpu_attention import Run, tables

pytestmark = pytest.mark.gpu


def near_zero(rng, w, dim):
    """Codes [tokens, dim] of values for which sum w v is small beside sum w |v|."""
    codes = rng.integers(0, 256, (200000, len(w)))
    codes = codes[((codes & 0x7F) < 0x70).all(1) & ((codes & 0x7F) >= 0x30).all(1)]
    v = ref.E4M3[codes]
    order = np.argsort(np.abs(v @ w) / (np.abs(v) @ w))[:dim]
    return codes[order].T.astype(np.uint8)


@pytest.mark.parametrize("q_heads", [2, 8, 20])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_outputs_that_cancel(dim, q_heads):
    rng = np.random.default_rng(dim + q_heads)
    lengths, heads, scale = [5, 29, 200, 150], 2, np.float32(0.7)
    pages, table = tables(rng, lengths, 64)
    c = ref.Cache(pages, 64, heads, dim, table)
    for which in range(2):
        c.codes[which][:] = 0
        c.scales[which][:] = 127
    for b, n in enumerate(lengths):
        for h in range(heads):
            for t in range(n):  # far below the five: e^-5.6
                c.codes[0][table[b, t // 64], h, t % 64, 0] = 0xD0
            five = rng.choice(n, 5, replace=False)
            keys = rng.integers(0x28, 0x43, 5)  # 0.25 .. 2.75
            codes = near_zero(rng, np.exp(float(scale) * ref.E4M3[keys]), dim)
            for i, t in enumerate(five):
                c.codes[0][table[b, t // 64], h, t % 64, 0] = keys[i]
                c.codes[1][table[b, t // 64], h, t % 64] = codes[i]
    q = np.zeros((len(lengths), q_heads, dim))
    q[:, :, 0] = 1.0
    r = Run(c, lengths, 1, q_heads, scale=scale, q=q).call()
    r.check()
    got = r.out.double().cpu().numpy().reshape(q.shape)
    for b, n in enumerate(lengths):
        k, _ = c.values(0, b, n)
        v, _ = c.values(1, b, n)
        w = np.exp(float(scale) * k[:, :, 0])
        want = np.einsum("th,thd->hd", w, v) / w.sum(0)[:, None]
        size = np.einsum("th,thd->hd", w, np.abs(v)) / w.sum(0)[:, None]
        for h in range(q_heads):
            at = h // (q_heads // heads)
            assert (np.abs(got[b, h] - want[at]) <= 2.0 ** -8 * np.abs(want[at]) + 2.0 ** -16 * size[at]).all()
    assert mx.mx_device_status() == 0
