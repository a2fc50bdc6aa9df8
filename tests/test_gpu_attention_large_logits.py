"""Logits far beyond 2^24, where binary32 has no halves: the tokens with the largest one share the row
evenly (others are hundreds below), under value scales that lie apart.

The logits of equal keys are equal in any arithmetic, so outputs are means of a few values: half a
BF16 step, 2^-8 relative, and 2^-20 of the values' size for binary32's sums.  A log-sum-exp is off by
the five roundings of a logit's scaling, 2^-21 relative."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests import decode_ref as ref
from tests.test_gpu_attention import Run, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length", [96, 6000])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("log2_size", [10.0, 24.0000055, 24.3, 25.0, 26.0000002, 26.7, 31.5, 60.2, 127.4])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_logits_share_the_row(length, dim, log2_size, sign):
    rng = np.random.default_rng(int(log2_size * 100) + dim)
    lengths, heads = [length, 50], 2
    pages, table = tables(rng, lengths, 32)
    c = ref.Cache(pages, 32, heads, dim, table)
    values = rng.integers(0, 256, c.codes[1].shape).astype(np.uint8)
    c.codes[1] = np.where((values & 0x7F) == 0x7F, 0x33, values).astype(np.uint8)
    c.scales[1] = rng.integers(127 - 20, 127 + 5, c.scales[1].shape).astype(np.uint8)
    c.scales[0][:] = 127
    c.codes[0][:] = 0
    # keys: 1 for the ones that share the row, 0.5 for the others (-1 and -2 for negative logits)
    c.codes[0][..., 0] = 0x30 if sign > 0 else 0xC0
    chosen = [sorted({*rng.choice(n, 4, replace=False), 0, n - 1}) for n in lengths]
    for b in range(2):
        for t in chosen[b]:
            c.codes[0][table[b, t // 32], :, t % 32, 0] = 0x38 if sign > 0 else 0xB8
    q = np.zeros((2, 4, dim))
    q[:, :, 0] = 1.0
    scale = np.float32(2.0 ** log2_size)
    r = Run(c, lengths, 1, 4, scale=scale, q=q).call()
    assert mx.mx_device_status() == 0
    got, lse = r.out.double().cpu().numpy().reshape(q.shape), r.lse.double().cpu().numpy().reshape(2, 4)
    assert np.isfinite(got).all()
    for b in range(2):
        v = c.values(1, b, lengths[b])[0][chosen[b]]
        want, size = v.mean(0), np.abs(v).mean(0)
        for h in range(4):
            err = np.abs(got[b, h] - want[h // 2])
            assert (err <= 2.0 ** -8 * np.abs(want[h // 2]) + 2.0 ** -20 * size[h // 2]).all()
        want = sign * float(scale) + np.log(len(chosen[b]))
        assert (np.abs(lse[b] - want) <= 2.0 ** -21 * (np.abs(want) + 1)).all()
