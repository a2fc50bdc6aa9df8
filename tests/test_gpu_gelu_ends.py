"""GELU far from zero: y where y > 0 and 0 where y < 0, up to the infinities; NaN stays NaN.
A bias of the type's lowest value switches an output off; y^2 is past binary32 from 1.8e19 on."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
import oracle
from block_scaled_fp4_bf16_gb300 import synth
from tests.gpu_helpers import dev_u8
from tests.test_gpu_few_tokens import FMTS, MX, NV, run_experts, run_linear, x_bits

pytestmark = pytest.mark.gpu

LOWEST = float(np.finfo(np.float32).min)
VALUES = [20.0, 63.0, 64.0, 65.0, 1e4, 1e10, 1.8e19, 1.9e19, 1e30, 3e38, -LOWEST, np.inf]
BIAS = np.array([s * v for v in VALUES for s in (1, -1)] + [0.0, np.nan], dtype=np.float32)
WANT = np.where(BIAS > 0, BIAS, np.where(np.isnan(BIAS), np.nan, 0.0))


def padded(n):
    b = np.zeros(n, np.float32)
    b[:len(BIAS)] = BIAS
    return b


def check(got, what):
    """got: rows of len(BIAS) outputs."""
    for row in got:
        assert np.array_equal(row, WANT.astype(np.float32).astype(row.dtype), equal_nan=True), (what, row)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,n,k", [(3, 96, 160), (20, 96, 160), (3, 8224, 8224), (20, 8224, 8224)])
def test_linear(fmt, tokens, n, k):
    class Zero:
        rows = n
    Zero.fmt = fmt
    dev = (torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda"),
           torch.full((mx.mx_scale_bytes(n, k, fmt, mx.MX_SCALE_TCGEN05),), 0x38 if fmt == NV else 127,
                      dtype=torch.uint8, device="cuda"),
           torch.ones(1, device="cuda") if fmt == NV else None)
    got = run_linear(x_bits(tokens, k, 1), Zero, bias=padded(n), gelu_on=True, dev=dev)
    check(got[:, :len(BIAS)], "linear")


@pytest.mark.parametrize("m", [32, 128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_gemm(fmt, m):
    n, k = 256, 256
    zero = lambda rows: torch.zeros((rows, k // 2), dtype=torch.uint8, device="cuda")  # noqa: E731
    one = lambda rows: torch.full((mx.mx_scale_bytes(rows, k, fmt, mx.MX_SCALE_TCGEN05),),  # noqa: E731
                                  0x38 if fmt == NV else 127, dtype=torch.uint8, device="cuda")
    bias, d = torch.from_numpy(padded(n)).cuda(), torch.full((m, n), 7.0, device="cuda")
    if fmt == MX:
        mx.mxfp4_gemm_ex(zero(m), one(m), zero(n), one(n), d, m, n, k, out_dtype=mx.MX_OUT_FP32, bias=bias,
                         gelu=True)
    else:
        ts = torch.ones(1, device="cuda")
        mx.nvfp4_gemm_ex(zero(m), one(m), zero(n), one(n), ts, ts, d, m, n, k, out_dtype=mx.MX_OUT_FP32,
                         bias=bias, gelu=True)
    check(d.cpu().numpy()[:, :len(BIAS)], "gemm")


def test_experts():
    """Gates of 2^66 and -2^66 (MXFP4 scales), up sums of 2^-60: y = 2^6 and 0."""
    n = 64
    gate, s = np.full((n, n // 2), 0, np.uint8), np.full((n, n // 32), 127, np.uint8)
    gate[:, 0] = np.where(np.arange(n) % 2, 0x0A, 0x02)  # code -1 or 1 of element 0
    gs, us = s.copy(), s.copy()
    gs[:, 0], us[:, 0] = 127 + 66, 127 - 60
    up, eye = np.zeros((n, n // 2), np.uint8), np.zeros((n, n // 2), np.uint8)
    up[:, 0] = 0x02
    eye[np.arange(n), np.arange(n) // 2] = np.where(np.arange(n) % 2, 0x20, 0x02)
    mats = [(dev_u8(c), dev_u8(oracle.scale_tile(q)), None) for c, q in ((gate, gs), (up, us), (eye, s))]

    class One:
        i = n
    One.moe = mx.moe_weights(MX, 1, n, n, *mats, mx.MX_ACT_GELU)
    x = np.zeros((2, n), np.float32)
    x[:, 0] = 1.0
    got = run_experts(One, synth.f32_to_bf16_bits(x), np.zeros((2, 1), np.int32), np.ones((2, 1), np.float32))
    assert (got == np.where(np.arange(n) % 2, 0.0, 2.0 ** 6)).all()
