"""mx_attention_bf16 where the lengths come to more than 2^36 tokens together: nothing is seen, and
mx_device_status says so."""
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests.gpu_helpers import check_guards, guarded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sequences,q_tokens", [(33, 1), (33, 5), (385, 1), (1000, 2), (4096, 1)])
def test_nothing_is_seen(dim, sequences, q_tokens):
    page, length = 1 << 20, 2 ** 31 - 1
    max_pages = 2048  # (room for the length)
    codes = [torch.full((page * dim,), 0x38, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((page // 32,), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = mx.kv_cache(codes[0], scales[0], codes[1], scales[1], 1, page, 1, dim)
    table = torch.zeros(sequences, max_pages, dtype=torch.int32, device="cuda")
    lengths = torch.full((sequences,), length, dtype=torch.int32, device="cuda")
    rows, cols = sequences * q_tokens, 2 * dim
    q = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    out, lse = guarded(rows * cols, torch.bfloat16, 5.0), guarded(rows * 2, torch.float32, 5.0)
    ws = guarded(mx.mx_attention_workspace_bytes(sequences, q_tokens, 2, cache))

    def call(window):
        mx.mx_attention_bf16(q, cols, 2, sequences, q_tokens, table, max_pages, lengths, cache, dim ** -0.5, window, out, cols,
                             lse, ws)
        return mx.mx_device_status()

    for _ in range(3):
        out.fill_(5.0)
        lse.fill_(5.0)
        assert call(0) == mx.MX_ERR_DEVICE_INDEX
        assert (out == 0).all() and torch.isneginf(lse).all()
        check_guards(out, lse, ws)
    # with a window the same lengths have few blocks: equal values and logits
    assert call(40) == 0
    assert (out == 1).all()
    want = dim ** 0.5 + torch.log(torch.tensor(40.0))
    assert ((lse.cpu() - want).abs() < 1e-4).all()
