"""The workspaces' sizes are 0 for sizes that the calls refuse (no GPU: the checks come
before the device)."""
import pytest

import block_scaled_fp4_bf16_gb300 as mx
from block_scaled_fp4_bf16_gb300 import build as _build

FAKE, GB = 0x7F0000000000, 1 << 30


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mx.lib()


@pytest.mark.parametrize("fmt,n,k", [(0, 1 << 20, 1 << 17), (1, 1 << 20, 1 << 16), (1, 32, 1 << 30),
                                     (0, 100, 8192), (0, 8192, 8200), (0, 1 << 31, 32)])
def test_linear(lib, fmt, n, k):
    ts = FAKE + 900 * GB if fmt == 1 else None
    assert lib.mx_linear_bf16(FAKE, 1, k, (k + 7) // 8 * 8, fmt, FAKE + 100 * GB, FAKE + 400 * GB, ts, n,
                              FAKE + 800 * GB, n, 0, None, None) == mx.MX_ERR_UNSUPPORTED_SHAPE
    assert mx.mx_linear_workspace_bytes(1, k, n, fmt) == 0


@pytest.mark.parametrize("hidden,inter", [(48, 128), (256, 100), (33, 33), (256, 1 << 31)])
def test_experts(lib, hidden, inter):
    m = [(FAKE + (1 + 2 * j) * GB, FAKE + (2 + 2 * j) * GB, None) for j in range(3)]
    moe = mx.moe_weights(mx.MX_FMT_MXFP4, 1, hidden, inter, *m)
    ld = (hidden + 7) // 8 * 8
    assert lib.mx_moe_experts_bf16(FAKE, 1, ld, FAKE + 10 * GB, FAKE + 11 * GB, 1, moe, FAKE + 12 * GB, ld,
                                   FAKE + 13 * GB, GB, None) == mx.MX_ERR_UNSUPPORTED_SHAPE
    assert mx.mx_moe_workspace_bytes(1, hidden, inter, 1) == 0
