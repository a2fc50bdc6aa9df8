"""SiLU of strongly negative gates, where exp(-g) nears and passes binary32's end while
silu(g) = -|g| exp(-|g|) does not, made visible by up sums of 2^100."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
import oracle
from block_scaled_fp4_bf16_gb300 import synth
from tests.gpu_helpers import dev_u8
from tests.test_gpu_few_tokens import FMTS, MX, assert_close, block, run_experts, ulp

pytestmark = pytest.mark.gpu

N = 64  # hidden and inter
X = [-12.0, -4.0, -1.0, -0.25, 1.0]
# the gate of a quarter of the rows each: 12 a + 4 b + c + d / 4
QUARTERS = [(6.0, 1.0, 4.0), (6.0, 3.0, 1.0), (6.0, 4.0, 0.0), (6.0, 4.0, 3.0)]
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def matrix(values, fmt, scale):
    """Device (codes, scales, tensor scale) of one expert's E2M1 values times a power of two."""
    code = np.array([E2M1.index(abs(v)) + (8 if v < 0 else 0) for v in values.ravel()]).reshape(values.shape)
    packed = (code[:, ::2] | code[:, 1::2] << 4).astype(np.uint8)
    s = np.full((len(values), values.shape[1] // block(fmt)), 127 + scale if fmt == MX else 0x38, np.uint8)
    ts = None if fmt == MX else torch.tensor([2.0 ** scale], dtype=torch.float32, device="cuda")
    return dev_u8(packed), dev_u8(oracle.scale_tile(s)), ts


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [1, 6, 12])
def test_strongly_negative_gates(fmt, tokens):
    gate, up = np.zeros((N, N)), np.zeros((N, N))
    for r in range(N):
        gate[r, :3] = QUARTERS[r // 16]
        gate[r, 3] = E2M1[r % 8] * (1 if r % 16 < 8 else -1)
    up[:, 4] = 1.0
    x = np.zeros((tokens, N))
    x[:, :5] = X
    moe = mx.moe_weights(fmt, 1, N, N, matrix(gate, fmt, 0), matrix(up, fmt, 100), matrix(np.eye(N), fmt, 0),
                         mx.MX_ACT_SILU)

    class Layer:
        i = N
    Layer.moe = moe
    got = run_experts(Layer, synth.f32_to_bf16_bits(x.astype(np.float32)), np.zeros((tokens, 1), np.int32),
                      np.ones((tokens, 1), np.float32))
    g, u = x @ gate.T, x @ up.T * 2.0 ** 100
    assert g.min() < -88.8 < -87 < g.max()
    h = g / (1.0 + np.exp(-g)) * u
    top = np.abs(h).reshape(tokens, -1, 16).max(2).repeat(16, 1)
    # expf and the quotient 2^-21, an exponential that is subnormal, the digits of h, a BF16 output
    tol = 2.0 ** -20 * np.abs(h) + 2.0 ** -149 * np.abs(g * u) + 2.0 ** -21 * top + ulp(h)
    assert_close(got, h, tol, "silu")
    assert (got != 0).all()
