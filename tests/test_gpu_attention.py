"""mx_attention_bf16 against the formula in binary64, with the error bound of
decode_ref.attention plus half a BF16 step (2^-8 relative) of each output."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests import decode_ref as ref
from tests.gpu_helpers import check_guards, guarded

pytestmark = pytest.mark.gpu


def filled(pages, page, heads, dim, table, seed, low=118, high=122):
    """A cache of random codes (no NaN) and scales of a spread."""
    c = ref.Cache(pages, page, heads, dim, table, seed)
    rng = np.random.default_rng(seed + 1)
    for which in range(2):
        c.codes[which] = ref.e4m3_round(np.clip(rng.normal(size=c.codes[which].shape) * 60, -448, 448))
        c.scales[which] = rng.integers(low, high, c.scales[which].shape).astype(np.uint8)
    return c


def tables(rng, lengths, page, extra=2):
    """(pages, table) of scattered pages, -1 behind each end."""
    used = [-(-max(int(n), 0) // page) for n in lengths]
    total = sum(used) + extra
    order = rng.permutation(total)
    table = np.full((len(lengths), max(1, max(used))), -1, np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return total, table


class Run:
    def __init__(self, cache, lengths, q_tokens, q_heads, window=0, scale=None, seed=0, pad=0, q=None):
        rng = np.random.default_rng(seed)
        self.c, self.lengths, self.n, self.h, self.window = cache, lengths, q_tokens, q_heads, window
        self.scale = np.float32(scale if scale is not None else cache.dim ** -0.5)
        rows = len(lengths) * q_tokens
        self.q = ref.bf16_round(rng.normal(size=(rows, q_heads, cache.dim))) if q is None else q
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.codes, self.scales = [dev(a) for a in cache.codes], [dev(a) for a in cache.scales]
        self.table, self.len = dev(cache.table), torch.tensor([int(n) for n in lengths], dtype=torch.int32, device="cuda")
        self.handle = mx.kv_cache(self.codes[0], self.scales[0], self.codes[1], self.scales[1], cache.pages,
                                  cache.page_tokens, cache.heads, cache.dim)
        cols = q_heads * cache.dim
        self.ld = cols + pad
        self.dq = torch.full((rows, self.ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.dq[:, :cols] = torch.from_numpy(self.q.reshape(rows, cols)).to("cuda", torch.bfloat16)
        self.body = guarded(rows * self.ld, torch.bfloat16, 5.0)
        self.out = self.body.view(rows, self.ld)
        self.lse = guarded(rows * q_heads, torch.float32, 5.0)
        self.ws = guarded(mx.mx_attention_workspace_bytes(len(lengths), q_tokens, q_heads, self.handle))

    def call(self, lse=True, stream=None):
        mx.mx_attention_bf16(self.dq, self.ld, self.h, len(self.lengths), self.n, self.table, self.table.shape[1],
                             self.len, self.handle, float(self.scale), self.window, self.out, self.ld,
                             self.lse if lse else None, self.ws, stream=stream)
        return self

    def check(self, status=0):
        assert mx.mx_device_status() == status
        check_guards(self.body, self.lse, self.ws)
        rows, cols = self.q.shape[0], self.h * self.c.dim
        most = self.c.table.shape[1] * self.c.page_tokens
        with np.errstate(invalid="ignore"):
            out, lse, e_out, e_lse = ref.attention(self.c, self.q, np.minimum(self.lengths, most), self.n, self.h,
                                                   float(self.scale), self.window)
        got = self.out[:, :cols].double().cpu().numpy().reshape(out.shape)
        got_lse = self.lse.double().cpu().numpy().reshape(lse.shape)
        assert np.array_equal(np.isnan(got), np.isnan(out))
        fine = ~np.isnan(out)
        assert (np.abs(got - out)[fine] <= (2.0 ** -8 * np.abs(out) + e_out + 1e-37)[fine]).all(), \
            (np.abs(got - out) / (2.0 ** -8 * np.abs(out) + e_out + 1e-37))[fine].max()
        assert np.array_equal(np.isneginf(got_lse), np.isneginf(lse))
        f = np.isfinite(lse)
        assert (np.abs(got_lse[f] - lse[f]) <= e_lse[f]).all()
        assert (self.out[:, cols:] == 5.0).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 7), (1, 16), (2, 17), (1, 64)])
def test_head_layouts(dim, heads, group):
    rng = np.random.default_rng(dim + heads + group)
    lengths = [1, 33, 200]
    pages, table = tables(rng, lengths, 64)
    Run(filled(pages, 64, heads, dim, table, 3), lengths, 1, heads * group, pad=8).call().check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("length", [0, 1, 2, 31, 32, 33, 63, 64, 65, 95, 96, 97, 1000])
def test_lengths(dim, length):
    rng = np.random.default_rng(length)
    lengths = [length, 7]
    pages, table = tables(rng, lengths, 32)
    Run(filled(pages, 32, 2, dim, table, 4), lengths, 1, 4).call().check()


@pytest.mark.parametrize("page", [32, 96, 256])
@pytest.mark.parametrize("q_tokens", [1, 2, 5, 16])
@pytest.mark.parametrize("window", [0, 1, 3, 32, 100])
def test_masks(page, q_tokens, window):
    rng = np.random.default_rng(page + q_tokens + window)
    lengths = [0, 1, 4, 17, 40, 160, 333]  # the first ones leave rows without anything
    pages, table = tables(rng, lengths, page)
    Run(filled(pages, page, 2, 64, table, 5), lengths, q_tokens, 6, window).call().check()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_more_rows_than_a_tile_and_drafts(dim):
    rng = np.random.default_rng(1)
    lengths = [300, 0, 9, 64]
    pages, table = tables(rng, lengths, 64)
    Run(filled(pages, 64, 2, dim, table, 6), lengths, 7, 2 * 9, 50).call().check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lengths", [[20000], [40000, 1, 300], [5] * 600])
def test_shares_of_workers(dim, lengths):
    """Rows that many workers share, and workers that have many rows."""
    rng = np.random.default_rng(2)
    pages, table = tables(rng, lengths, 128)
    Run(filled(pages, 128, 1, dim, table, 7), lengths, 1, 2).call().check()


def test_uneven_weights_and_scales():
    """Logits of a wide range, scales far apart in keys and values."""
    rng = np.random.default_rng(3)
    lengths = [700, 64]
    pages, table = tables(rng, lengths, 32)
    c = filled(pages, 32, 2, 128, table, 8, 100, 134)
    Run(c, lengths, 2, 8, scale=0.01).call().check()
    # values of the block with the largest weight 2^60 below those of blocks with none to speak of
    c.scales[0][:] = 119
    c.scales[1][:] = 180
    t0 = table[0, 3]
    c.scales[1][t0] = 120
    c.codes[0][t0, :, 5] = c.codes[0][t0, :, 5] & 0x7F
    q = np.abs(ref.bf16_round(rng.normal(size=(4, 8, 128))))
    c.codes[0][t0, :, 5] = 0x70  # 256: far ahead of the others
    Run(c, lengths, 2, 8, scale=0.5, q=q).call().check()


@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -30, 2.0 ** 100])
def test_queries_of_any_size(size):
    rng = np.random.default_rng(4)
    lengths = [70, 5]
    pages, table = tables(rng, lengths, 32)
    q = ref.bf16_round(rng.normal(size=(2, 4, 64)) * size)
    q[0, 0, :32] *= 2.0 ** -20
    q[1, 1] = 0.0
    c = filled(pages, 32, 2, 64, table, 9)
    Run(c, lengths, 1, 4, scale=np.float32(0.1 / size), q=ref.bf16_round(q)).call().check()


def test_negative_scale_and_equal_logits():
    rng = np.random.default_rng(4)
    lengths = [130, 64]
    pages, table = tables(rng, lengths, 64)
    c = filled(pages, 64, 1, 64, table, 9)
    Run(c, lengths, 1, 3, scale=-0.2).call().check()
    Run(c, lengths, 1, 3, scale=0.0).call().check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_tokens,window", [(1, 0), (4, 0), (4, 40), (1, 33)])
def test_nan_where_a_row_does_not_see_it(dim, q_tokens, window):
    """Behind the end, before the window, and in tokens that only later queries see."""
    rng = np.random.default_rng(5)
    lengths = [75, 64, 3]
    pages, table = tables(rng, lengths, 64)
    c = filled(pages, 64, 2, dim, table, 10)
    for b, n in enumerate(lengths):
        for p in range(c.table.shape[1]):
            page = table[b, p]
            if page < 0:
                continue
            for t in range(64):
                token = p * 64 + t
                if token >= n or (window and token <= n - q_tokens - window):
                    c.codes[0][page, :, t] = 0x7F
                    c.codes[1][page, :, t] = 0xFF
    Run(c, lengths, q_tokens, 4, window).call().check()
    # seen by the last query only (keys), and a value's channel
    page = table[0, 74 // 64]
    c.codes[1][page, 1, 74 % 64, 9] = 0x7F
    r = Run(c, lengths, q_tokens, 4, window).call()
    r.check()
    got = r.out.double().cpu().numpy().reshape(-1, 4, dim)
    assert np.isnan(got[q_tokens - 1, 2:, 9]).all() and np.isnan(got).sum() == 2
    c.codes[1][page, 1, 74 % 64, 9] = 0
    c.codes[0][page, 0, 74 % 64, 1] = 0xFF
    r = Run(c, lengths, q_tokens, 4, window).call()
    r.check()
    got = r.out.double().cpu().numpy().reshape(-1, 4, dim)
    assert np.isnan(got[q_tokens - 1, :2]).all() and np.isnan(got).sum() == 2 * dim


def test_infinite_queries_stay_in_their_row():
    rng = np.random.default_rng(6)
    lengths = [90, 40]
    pages, table = tables(rng, lengths, 64)
    c = filled(pages, 64, 2, 128, table, 11)
    clean = Run(c, lengths, 2, 4).call()
    q = clean.q.copy()
    q[1, 2, 7] = np.inf
    q[2, 0, 0] = np.nan
    dirty = Run(c, lengths, 2, 4, q=q).call()
    torch.cuda.synchronize()
    a, b = (r.out.float().cpu().numpy().reshape(4, 4, 128) for r in (clean, dirty))
    bad = np.zeros_like(a, bool)
    bad[1, 2] = bad[2, 0] = True
    assert np.array_equal(a[~bad], b[~bad]) and np.isnan(b[bad]).all()


def test_pages_and_lengths_out_of_range():
    rng = np.random.default_rng(7)
    lengths = [200, 100, 128]
    pages, table = tables(rng, lengths, 32)
    table[0, 2], table[1, 0], table[1, 3] = -1, pages, 2 ** 31 - 1
    c = filled(pages, 32, 2, 64, table, 12)
    Run(c, lengths, 2, 4).call().check(mx.MX_ERR_DEVICE_INDEX)
    lengths = [32 * 7 + 1, -3, 64]
    table[0] = np.arange(7)
    c = filled(pages, 32, 2, 64, np.abs(table) % pages, 12)
    Run(c, lengths, 1, 4).call().check(mx.MX_ERR_DEVICE_INDEX)


def test_without_lse_and_the_same_bits_again():
    rng = np.random.default_rng(8)
    lengths = [3000, 17, 800]
    pages, table = tables(rng, lengths, 64)
    r = Run(filled(pages, 64, 4, 128, table, 13), lengths, 1, 16).call()
    first = r.out.clone()
    r.ws.fill_(0xFF)
    r.lse.fill_(5.0)
    r.call(lse=False)
    assert torch.equal(first, r.out) and (r.lse == 5.0).all()


def test_shared_pages():
    """Sequences that share their first pages read the same tokens."""
    rng = np.random.default_rng(9)
    table = np.array([[0, 1, 2], [0, 1, 3], [0, 0, 0]], np.int32)
    c = filled(4, 32, 2, 64, table, 14)
    Run(c, [96, 80, 70], 1, 4).call().check()


def test_offsets_past_32_bits():
    """A pool whose codes take more than 2^32 bytes: its last pages."""
    page, heads, dim = 1024, 8, 256
    pages = 2 ** 32 // (page * heads * dim) + 3
    codes = [torch.zeros(pages * heads * page * dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages * heads * page // 32,), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = mx.kv_cache(codes[0], scales[0], codes[1], scales[1], pages, page, heads, dim)
    n = 300
    k = torch.randn(n, heads * dim, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    v = torch.randn(n, heads * dim, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(torch.bfloat16)
    q = torch.randn(1, heads * dim, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(torch.bfloat16)
    out = []
    for at in (0, pages - 1):
        table = torch.tensor([[at]], dtype=torch.int32, device="cuda")
        lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
        mx.mx_kv_append_bf16(k, heads * dim, v, heads * dim, n, None, table, 1, lengths, 1, cache)
        y = torch.empty_like(q)
        ws = torch.empty(mx.mx_attention_workspace_bytes(1, 1, heads, cache), dtype=torch.uint8, device="cuda")
        mx.mx_attention_bf16(q, heads * dim, heads, 1, 1, table, 1, lengths, cache, dim ** -0.5, 0, y, heads * dim, None, ws)
        out.append(y)
    assert torch.equal(out[0], out[1]) and float(out[0].float().abs().max()) > 0
    p = heads * page * dim
    assert torch.equal(codes[0][:p], codes[0][-p:]) and int(codes[1][p:-p].max()) == 0
