"""mx_attention_workspace_bytes asks for what the kernels may write, and no more: for each of at most 160
CTAs where it goes on and two parts, and a part for each warp (no GPU).  That what they write
stays within is seen by the guards around the workspace in the GPU tests."""
import ctypes

import pytest

import block_scaled_fp4_bf16_gb300 as mx
from block_scaled_fp4_bf16_gb300 import build as _build


def cache(dim, heads=2):
    return mx.mx_kv_cache(None, None, None, None, 10, 64, heads, dim)


@pytest.mark.parametrize("dim,rows,part_rows,warps", [
    (64, 1, 1, 16), (64, 8, 8, 16), (64, 9, 9, 12), (64, 17, 16, 12), (64, 128, 16, 12), (128, 3, 3, 12), (128, 8, 8, 12), (128, 64, 8, 12),
    (256, 1, 1, 6), (256, 8, 8, 6), (256, 16, 8, 6)])
def test_size(dim, rows, part_rows, warps):
    _build.build()
    part = part_rows * dim + -(-3 * part_rows // 4) * 4  # sums, two maxima and a weight a row
    want = 160 * 16 + 160 * (2 + warps) * part * 4
    lib = mx.lib()
    for q_tokens, group in ((1, rows), (rows, 1), (2, rows // 2)):
        if q_tokens <= mx.MX_ATTENTION_MAX_QUERY and 1 <= group <= 64 and q_tokens * group == rows:
            assert lib.mx_attention_workspace_bytes(5, q_tokens, 2 * group, ctypes.byref(cache(dim))) == want
