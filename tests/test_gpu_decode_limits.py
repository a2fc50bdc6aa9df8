"""The decoding step's calls at the ends of their ranges: offsets past 32 bits, the most rows, heads and
sequences.  Each is compared, bit for bit, with calls of ordinary sizes (which other tests compare with
the formulas) or with the definition."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests.test_gpu_attention import Run, filled, tables

pytestmark = pytest.mark.gpu

T, LD = (1 << 20) + 3, 4608  # T * LD elements are more than 2^32


def wide(cols, seed=None):
    """[T, cols] as columns 128 .. 128 + cols of rows of LD."""
    rows = torch.empty(T, LD, dtype=torch.bfloat16, device="cuda")
    v = rows[:, 128:128 + cols]
    if seed is not None:
        v.normal_(generator=torch.Generator("cuda").manual_seed(seed))
    return v


def norm_of():
    dim = 64
    w = [torch.linspace(0.5, 1.5, dim, device="cuda").to(torch.bfloat16) for _ in range(2)]
    return mx.qk_norm(2, 1, dim, *w, 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float32, device="cuda") / dim))


def test_norm_and_rotation_of_rows_past_32_bits():
    norm, cols = norm_of(), 192
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    x, y = wide(cols, 1), wide(cols)
    mx.mx_qk_norm_rope_bf16(x, LD, x[:, 128:], LD, T, pos, norm, y, LD, y[:, 128:], LD)
    c = x.contiguous()
    mx.mx_qk_norm_rope_bf16(c, cols, c[:, 128:], cols, T, pos, norm, c, cols, c[:, 128:], cols)
    assert torch.equal(y, c)
    assert mx.mx_device_status() == 0


def test_gradients_of_rows_past_32_bits():
    norm, cols = norm_of(), 192
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    x, dy, dx = wide(cols, 1), wide(cols, 2), wide(cols)
    ws = torch.empty(mx.mx_qk_norm_rope_backward_workspace_bytes(T, norm), dtype=torch.uint8, device="cuda")
    dw = torch.empty(2, 2, 64, device="cuda")
    mx.mx_qk_norm_rope_backward_bf16(x, LD, x[:, 128:], LD, dy, LD, dy[:, 128:], LD, T, pos, norm, dx, LD, dx[:, 128:], LD,
                                     dw[0, 0], dw[0, 1], ws)
    cx, cy = x.contiguous(), dy.contiguous()
    out = torch.empty_like(cx)
    mx.mx_qk_norm_rope_backward_bf16(cx, cols, cx[:, 128:], cols, cy, cols, cy[:, 128:], cols, T, pos, norm, out, cols,
                                     out[:, 128:], cols, dw[1, 0], dw[1, 1], ws)
    assert torch.equal(dx, out) and torch.equal(dw[0], dw[1])
    assert mx.mx_device_status() == 0


def test_append_of_rows_past_32_bits_and_of_the_largest_page():
    page = 1 << 20
    kv = wide(128, 3)
    compact = kv.contiguous()
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([T], dtype=torch.int32, device="cuda")
    pools = []
    for rows, ld in ((kv, LD), (compact, 128)):
        pool = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (2 * page * 64, 2 * page // 32) * 2]
        mx.mx_kv_append_bf16(rows, ld, rows[:, 64:], ld, T, None, table, 2, lengths, 1, mx.kv_cache(*pool, 2, page, 1, 64))
        pools.append(pool)
    assert all(torch.equal(a, b) for a, b in zip(*pools))
    assert int(pools[0][0][:3 * 64].max()) > 0 and int(pools[0][0][3 * 64:page * 64].max()) == 0  # (page 0: the last three)
    assert int(pools[0][1].count_nonzero()) == page // 32 + 1
    assert mx.mx_device_status() == 0


def test_attention_of_the_most_heads_and_queries():
    """1024 key heads of 64 x 16 rows, which are copies of four; a block each, so that no sum is shared out."""
    kinds, dim, n, length = 4, 64, 16, 32
    c = filled(1, 32, kinds, dim, np.zeros((1, 1), np.int32), 3)
    small = Run(c, [length], n, 64 * kinds).call()
    big = filled(1, 32, 1, dim, np.zeros((1, 1), np.int32), 3)
    big.heads = 1024
    big.codes = [np.tile(v, (1, 256, 1, 1)) for v in c.codes]
    big.scales = [np.tile(v, (1, 256, 1)) for v in c.scales]
    large = Run(big, [length], n, 64 * 1024, q=np.tile(small.q, (1, 256, 1))).call()
    assert mx.mx_device_status() == 0
    want = small.out.view(n, 1, -1).expand(n, 256, -1).reshape(n, -1)
    assert torch.equal(large.out, want)
    assert torch.equal(large.lse.view(n, 256, -1), small.lse.view(n, 1, -1).expand(n, 256, -1))


@pytest.mark.parametrize("dim", [64, 256])
def test_attention_of_the_most_sequences(dim):
    rng = np.random.default_rng(dim)
    lengths = rng.integers(0, 70, 4096) * (rng.random(4096) < 0.7)
    pages, table = tables(rng, lengths, 32)
    Run(filled(pages, 32, 1, dim, table, 5), lengths, 1, 2).call().check()


def test_sampling_of_the_most_rows():
    rows, vocab = 1 << 20, 9
    x = torch.randn(rows, vocab, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    u = torch.rand(rows, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    ids = torch.empty(rows, dtype=torch.int32, device="cuda")
    prob = torch.empty(rows, device="cuda")
    greedy = torch.where(torch.arange(rows, device="cuda") % 2 == 0, 0.0, 1.0)
    one = torch.where(torch.arange(rows, device="cuda") % 2 == 0, 0, 1).to(torch.int32)
    mx.mx_sample(x, rows, vocab, vocab, mx.MX_OUT_FP32, greedy, one, None, None, u, ids, prob)
    assert torch.equal(ids.long(), x.argmax(1)) and (prob == 1).all()
    # without filters: the definition in binary64 (a uniform number within 2^-30 of a border may go either way)
    mx.mx_sample(x, rows, vocab, vocab, mx.MX_OUT_FP32, None, None, None, None, u, ids, prob)
    p = torch.softmax(x.double(), 1)
    upto = p.cumsum(1)
    want = (upto <= u.double()[:, None]).sum(1).clamp(max=vocab - 1)
    near = (upto - u.double()[:, None]).abs().min(1).values < 2.0 ** -30
    assert (near | (ids == want)).all() and int(near.sum()) < 100
    got = p.gather(1, ids.long()[:, None])[:, 0]
    assert ((prob.double() - got).abs() <= 2.0 ** -22 * got).all()
    assert mx.mx_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_past_32_bits(dtype):
    rows, vocab, ld = 600, 20001, (1 << 23) + 5
    x = torch.empty(rows * ld, dtype=dtype, device="cuda").view(rows, ld)[:, :vocab]
    x.normal_(std=3.0, generator=torch.Generator("cuda").manual_seed(1))
    u = torch.rand(rows, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    top_k = torch.arange(rows, dtype=torch.int32, device="cuda") % 7 * 20
    top_p = torch.linspace(0.3, 1.2, rows, device="cuda")
    code = mx.MX_OUT_FP32 if dtype is torch.float32 else mx.MX_OUT_BF16
    out = []
    for v, step in ((x, ld), (x.contiguous(), vocab)):
        ids, prob = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
        mx.mx_sample(v, rows, vocab, step, code, None, top_k, top_p, None, u, ids, prob)
        out.append((ids, prob))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert int(out[0][0].min()) >= 0 and mx.mx_device_status() == 0
