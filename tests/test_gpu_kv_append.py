"""mx_kv_append_bf16: codes and scales byte for byte those of the definition, everything else of the
pool as it was."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests import decode_ref as ref
from tests.gpu_helpers import check_guards, guarded

pytestmark = pytest.mark.gpu


class Device:
    """A reference cache's copy on the GPU, between guards."""

    def __init__(self, cache):
        self.c = cache

        def put(a):
            t = guarded(a.size)
            t.copy_(torch.from_numpy(a.reshape(-1)))
            return t

        self.codes, self.scales = [put(a) for a in cache.codes], [put(a) for a in cache.scales]
        self.table = torch.from_numpy(cache.table).cuda()
        self.handle = mx.kv_cache(self.codes[0], self.scales[0], self.codes[1], self.scales[1], cache.pages,
                                  cache.page_tokens, cache.heads, cache.dim)

    def append(self, k, v, counts, lengths, starts=True, ld=None, stream=None):
        """k, v: binary64 [tokens, heads, dim] that are BF16 values."""
        cols, t = self.c.heads * self.c.dim, k.shape[0]
        ld = ld or cols
        rows = []
        for x in (k, v):
            full = torch.full((max(t, 1), ld), float("nan"), dtype=torch.bfloat16, device="cuda")
            full[:t, :cols] = torch.from_numpy(x.reshape(t, cols)).to("cuda", torch.bfloat16)
            rows.append(full)
        s = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda() if starts else None
        n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        mx.mx_kv_append_bf16(rows[0], ld, rows[1], ld, t, s, self.table, self.table.shape[1], n, len(counts), self.handle,
                             stream=stream)
        torch.cuda.synchronize()

    def check(self):
        check_guards(*self.codes, *self.scales)
        for which in range(2):
            assert np.array_equal(self.scales[which].cpu().numpy(), self.c.scales[which].reshape(-1)), "scales"
            assert np.array_equal(self.codes[which].cpu().numpy(), self.c.codes[which].reshape(-1)), "codes"


def both(cache, rng, counts, lengths, spread=2.0, edit=None, **kw):
    t = int(np.sum(counts))
    new = [ref.bf16_round(rng.normal(size=(t, cache.heads, cache.dim)) * np.exp(spread * rng.normal(size=(t, 1, 1))))
           for _ in range(2)]
    if edit:
        edit(new)
    d = kw.pop("device", None) or Device(cache)
    d.append(new[0], new[1], counts, lengths, **kw)
    with np.errstate(invalid="ignore"):
        cache.append(new, counts, lengths)
    d.check()
    assert mx.mx_device_status() == 0
    return d


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [32, 64, 96])
def test_prompts_then_tokens(dim, page):
    rng = np.random.default_rng(dim + page)
    cache = ref.Cache(20, page, 2, dim, rng.permutation(20)[:18].reshape(3, 6), 1)
    lengths = np.array([1, 45, 100])
    d = both(cache, rng, list(lengths), list(lengths))
    for _ in range(3):  # one token each, without and with starts
        lengths = lengths + 1
        both(cache, rng, [1, 1, 1], list(lengths), device=d, starts=False)
    more = [31, 0, 33]
    lengths = lengths + more
    both(cache, rng, more, list(lengths), device=d)
    lengths = lengths + 3
    both(cache, rng, [3, 3, 3], list(lengths), device=d, starts=False)


@pytest.mark.parametrize("offset", [0, 1, 30, 31])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 34, 65])
def test_any_place_in_a_block(offset, n):
    rng = np.random.default_rng(offset * 100 + n)
    cache = ref.Cache(5, 64, 1, 64, [[3, 1, 4, 0]], 2)
    d = Device(cache)
    if offset:
        both(cache, rng, [offset], [offset], device=d)
    both(cache, rng, [n], [offset + n], device=d)
    both(cache, rng, [n], [offset + 2 * n], device=d, starts=False) if offset + 2 * n <= 256 else None


def test_strides_and_many_sequences():
    rng = np.random.default_rng(0)
    n = 300
    cache = ref.Cache(n, 32, 3, 64, rng.permutation(n).reshape(n, 1), 3)
    counts = rng.integers(0, 3, n)
    both(cache, rng, list(counts), list(counts + rng.integers(0, 20, n)), ld=3 * 64 + 24)


def test_scales_at_their_borders():
    rng = np.random.default_rng(0)
    top = [448.0, 450.0, 1.75 * 2.0 ** -10, 1.7578125 * 2.0 ** -10, 0.0, 3.0e38, 2.0 ** -133, 1.75 * 2.0 ** -119,
           1.7578125 * 2.0 ** -119, 2.0 ** -126]

    def edit(new):
        for i, v in enumerate(top):
            for x in new:
                x[32 * i:32 * i + 32] *= 0.0 if v == 0 else min(1.0, v) * 2.0 ** -30
                x[32 * i:32 * i + 32] = ref.bf16_round(x[32 * i:32 * i + 32])
                x[32 * i + 5, 0, 7] = -v
    n = 32 * len(top)
    cache = ref.Cache(10, 32, 1, 64, [list(range(10))], 4)
    both(cache, rng, [n], [n], spread=0.0, edit=edit)


def test_infinities_and_nan_become_nan_and_leave_the_scale():
    rng = np.random.default_rng(0)

    def edit(new):
        new[0][3, 0, 5], new[0][3, 1, 6], new[1][40, 0, 0] = np.inf, np.nan, -np.inf
        new[1][32:40] = np.nan
        new[1][41:64] = np.inf
    cache = ref.Cache(2, 64, 2, 64, [[1]], 5)
    d = both(cache, rng, [64], [64], edit=edit)
    both(cache, rng, [10], [64], device=d)  # over them, from the middle of the block


def test_a_block_of_nothing_finite_has_the_least_scale():
    rng = np.random.default_rng(0)

    def edit(new):
        new[1][:] = np.where(rng.random(new[1].shape) < 0.5, np.inf, np.nan)
    cache = ref.Cache(1, 32, 2, 64, [[0]], 5)
    both(cache, rng, [32], [32], edit=edit)
    assert (cache.scales[1] == 0).all() and (cache.scales[0] > 0).all()


def test_scales_that_grow_again_and_again():
    rng = np.random.default_rng(0)
    cache = ref.Cache(1, 32, 1, 128, [[0]], 6)
    d = Device(cache)
    for i in range(32):
        def edit(new, i=i):
            for x in new:
                x *= 2.0 ** (i // 2)
        both(cache, rng, [1], [i + 1], spread=0.3, edit=edit, device=d, starts=False)


def test_empty_slots_and_rows_before_the_beginning():
    rng = np.random.default_rng(0)
    cache = ref.Cache(6, 64, 2, 64, [[0, 1], [2, 3], [4, 5]], 7)
    both(cache, rng, [4, 4, 4], [0, 2, 50], starts=False)  # (the second: two rows have no position)
    both(cache, rng, [0, 40, 0], [0, 20, 50])


def test_pages_and_lengths_out_of_range_are_left_out_and_reported():
    rng = np.random.default_rng(0)
    cache = ref.Cache(4, 32, 1, 64, [[0, -1], [4, 1], [2, 3]], 8)
    d = Device(cache)
    new = [ref.bf16_round(rng.normal(size=(66, 1, 64))) for _ in range(2)]
    d.append(new[0], new[1], [33, 33, 0], [33, 64, 0])
    cache.append(new, [33, 33, 0], [33, 64, 0])
    d.check()
    assert mx.mx_device_status() == mx.MX_ERR_DEVICE_INDEX
    # beyond the table's row: 65 of 64 tokens
    new = [x[:3] for x in new]
    d.append(new[0], new[1], [0, 0, 3], [0, 0, 66])
    cache.append(new, [0, 0, 3], [0, 0, 66])
    d.check()
    assert mx.mx_device_status() == mx.MX_ERR_DEVICE_INDEX
    assert mx.mx_device_status() == 0


@pytest.mark.parametrize("starts", [[0, 5, 3, 6], [-1, 2, 3, 6], [0, 2, 4, 7], [0, 2, 9, 6]])
def test_starts_out_of_order_are_left_out_and_reported(starts):
    cache = ref.Cache(3, 32, 1, 64, [[0], [1], [2]], 9)
    d = Device(cache)
    x = torch.ones(6, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")
    n = torch.tensor([10, 10, 10], dtype=torch.int32, device="cuda")
    mx.mx_kv_append_bf16(x, 64, x, 64, 6, s, d.table, 1, n, 3, d.handle)
    assert mx.mx_device_status() == mx.MX_ERR_DEVICE_INDEX
    check_guards(*d.codes, *d.scales)


def test_nothing_to_store():
    cache = ref.Cache(1, 32, 1, 64, [[0]], 9)
    d = Device(cache)
    x = torch.ones(1, 64, dtype=torch.bfloat16, device="cuda")
    n = torch.tensor([1], dtype=torch.int32, device="cuda")
    mx.mx_kv_append_bf16(x, 64, x, 64, 0, None, d.table, 1, n, 1, d.handle)
    mx.mx_kv_append_bf16(x, 64, x, 64, 1, None, d.table, 1, n, 0, d.handle)
    d.check()
