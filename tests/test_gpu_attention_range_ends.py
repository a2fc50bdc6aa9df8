"""Logits of ordinary size whose factors lie at the ends of binary32's range: the scale, the queries'
and the keys' powers of two (tolerances: tests/decode_ref.attention), and logits of 0 beside others that leave it."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests import decode_ref as ref
from tests.test_gpu_attention import Run, filled, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("scale,query,key", [
    (3.4028234e38, 2.0 ** -120, -10), (3.0e38, 2.0 ** -120, -10), (-2.9e38, 2.0 ** -120, -10), (3.0e38, 2.0 ** -20, -110),
    (2.0 ** 127, 2.0 ** -128, -2),
    (2.0 ** 126, 2.0 ** -131, 2), (2.0 ** 10, 2.0 ** -130, 114), (2.0 ** -100, 2.0 ** -30, 120), (2.0 ** -126, 2.0 ** 120, 2),
    (2.0 ** -130, 2.0 ** 10, 114), (2.0 ** -140, 2.0 ** 110, 22), (2.0 ** 100, 2.0 ** 20, -126), (1.0, 2.0 ** 115, -125),
    (1.0, 2.0 ** -122, 115)])
def test_ordinary_logits(dim, scale, query, key):
    """scale * query * key = 2^-8 or so; codes are some 2^6, a sum of products of `dim` channels 2^9 or more."""
    rng = np.random.default_rng(dim)
    lengths = [300, 33, 2]
    pages, table = tables(rng, lengths, 32)
    c = filled(pages, 32, 2, dim, table, 15)
    c.scales[0] = (127 + key + rng.integers(0, 2, c.scales[0].shape)).astype(np.uint8)
    q = ref.bf16_round(rng.normal(size=(6, 4, dim)) * query)
    q[1, 1] = 0.0
    q[2, 2, 1:] = 0.0
    assert np.abs(q).max() > query
    Run(c, lengths, 2, 4, scale=np.float32(scale), q=q).call().check()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_logits_of_zero_stay_zero(dim):
    """Tokens whose keys have nothing where the query has: 0, and the others far below (or past) binary32's least."""
    rng = np.random.default_rng(dim)
    lengths = [100, 40]
    pages, table = tables(rng, lengths, 32)
    c = filled(pages, 32, 1, dim, table, 16)
    c.scales[0][:] = 254
    c.codes[0][..., 0] = 0xB8  # -1
    kept = [[3, 50, 99], [39]]
    for b in range(2):
        for t in kept[b]:
            c.codes[0][table[b, t // 32], 0, t % 32, 0] = 0
    q = np.zeros((2, 2, dim))
    q[:, :, 0] = 2.0 ** 120
    r = Run(c, lengths, 1, 2, scale=1.0, q=q).call()
    assert mx.mx_device_status() == 0
    got, lse = r.out.double().cpu().numpy().reshape(q.shape), r.lse.cpu().numpy().reshape(2, 2)
    for b in range(2):
        v = c.values(1, b, lengths[b])[0][kept[b], 0]
        assert (np.abs(got[b] - v.mean(0)) <= 2.0 ** -8 * np.abs(v.mean(0)) + 2.0 ** -20 * np.abs(v).mean(0)).all()
        assert np.abs(lse[b] - np.log(len(kept[b]))).max() <= 2.0 ** -21
    # (a query of zeros, too)
    r = Run(c, lengths, 1, 2, scale=3.0e38, q=np.zeros_like(q)).call()
    r.check()
    assert torch.isfinite(r.out).all()
