"""mx_kv_append_bf16 with starts that are out of order or range: those sequences are left out, byte
for byte, and the others stored."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests import decode_ref as ref
from tests.test_gpu_kv_append import Device

pytestmark = pytest.mark.gpu


def run(starts, tokens, lengths, stored, dim=64, heads=3):
    """Appends over a pool of random bytes; `stored`: the sequences that are."""
    rng = np.random.default_rng(len(starts) + tokens)
    pages = -(-max(lengths) // 32)
    cache = ref.Cache(len(lengths) * pages + 1, 32, heads, dim, rng.permutation(len(lengths) * pages).reshape(len(lengths), pages), 9)
    d = Device(cache)
    new = [ref.bf16_round(rng.normal(size=(tokens, heads, dim)) * np.exp(2 * rng.normal(size=(tokens, 1, 1)))) for _ in range(2)]
    rows = [torch.from_numpy(x.reshape(tokens, heads * dim)).to("cuda", torch.bfloat16) for x in new]
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    ld = heads * dim
    mx.mx_kv_append_bf16(rows[0], ld, rows[1], ld, tokens, s, d.table, pages, n, len(lengths), d.handle)
    for b in stored:
        s0, s1 = starts[b], starts[b + 1]
        counts = [0] * len(lengths)
        counts[b] = s1 - s0
        cache.append([x[s0:s1] for x in new], counts, lengths)
    d.check()
    whole = len(stored) == len(lengths)
    assert mx.mx_device_status() == (0 if whole else mx.MX_ERR_DEVICE_INDEX)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("starts,stored", [
    ([0, 5, 3, 6], [0, 2]), ([-1, 2, 3, 6], [1, 2]), ([0, 2, 4, 7], [0, 1]), ([0, 2, 9, 6], [0]), ([0, 2, 2, 6], [0, 1, 2]),
    ([6, 5, 4, 3], []), ([0, -2, 4, 6], [2])])
def test_the_others_are_stored(starts, stored, dim):
    run(starts, 6, [10, 40, 33], stored, dim)


def test_long_ones_beside_bad_ones():
    run([0, 100, 90, 230, 300], 260, [100, 50, 200, 80], [0, 2])
    run([0, 70, 71, 600, 200], 200, [130, 1, 64, 64], [0, 1])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_slots_of_two_sequences(dim):
    """Behind starts that descend, a sequence may share slots with an earlier one: it is left out as a whole."""
    run([0, 90, 0, 64], 100, [100, 20, 70], [0, 2], dim)
    run([0, 100, 0, 64], 100, [100, 20, 70], [0], dim)
    run([0, 1000, 0, 64, 1000, 1000], 1000, [1000, 20, 70, 950, 20], [0, 4], dim)
    run([0, 30, 400, 100, 100, 390], 400, [40, 380, 64, 80, 290], [0, 1], dim)
