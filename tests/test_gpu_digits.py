"""The products on FP4 digits by the accuracy that the header states: to within 2^-22 of a
block's largest (tests/digits.py), at random values and where nothing but the low digits of
x or of the hidden values reaches the outputs.  The tolerances tell seven digits from eight
(test_digits_cpu.py)."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
import oracle
from block_scaled_fp4_bf16_gb300 import synth
from tests import digits as d
from tests.gpu_helpers import bf16_bits_to_f64, check_guards, dev_bf16, dev_u8, guarded
from tests.test_digits_cpu import low_linear
from tests.test_gpu_few_tokens import FMTS, NV, SIZES, Layer, assert_close, choice, gelu, run_experts, x_bits

pytestmark = pytest.mark.gpu


def device(values, fmt):
    codes, scales = d.unpacked_tensors(values, fmt)
    ts = torch.ones(1, dtype=torch.float32, device="cuda") if fmt == NV else None
    return dev_u8(codes), dev_u8(oracle.scale_tile(scales)), ts


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [1, 3, 4, 6, 8, 12, 40, 64])
def test_low_digits_of_x_and_h(fmt, tokens):
    c = d.LowDigits(tokens, 601)

    class One:
        i = c.n
    One.moe = mx.moe_weights(fmt, 1, c.k, c.n, *(device(m, fmt) for m in (c.gate, c.up, c.down)))
    got = run_experts(One, synth.f32_to_bf16_bits(c.x.astype(np.float32)), np.zeros((tokens, 1), np.int32),
                      np.ones((tokens, 1), np.float32))
    y, tol = d.expert(c.x, c.gate, c.up, c.down, fmt)
    assert_close(got, y, tol + d.ulp(y), "low digits")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", [mx.MX_ACT_SILU, mx.MX_ACT_GELU])
@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k", SIZES)
def test_experts_by_the_stated_accuracy(fmt, act, tokens, hidden, inter, experts, top_k):
    layer = Layer(experts, hidden, inter, fmt, act, 611)
    bits = x_bits(tokens, hidden, 612)
    ids, w = choice(tokens, experts, top_k, 613)
    x, f = bf16_bits_to_f64(bits), d.silu if act == mx.MX_ACT_SILU else gelu
    y, tol, s = (np.zeros((tokens, hidden)) for _ in range(3))
    for e in range(experts):
        at = np.argwhere(ids == e)
        if len(at) == 0:
            continue
        z, dz = d.expert(x[at[:, 0]], layer.gate.w[e].value, layer.up.w[e].value, layer.down.w[e].value, fmt, f)
        for (t, j), zt, dt in zip(at, z, dz):
            y[t] += w[t, j] * zt
            tol[t] += w[t, j] * dt
            s[t] += w[t, j] * np.abs(zt)
    assert_close(run_experts(layer, bits, ids, w), y, tol + 2.0 ** -20 * s + d.ulp(y), "experts")


# with a workspace; and without one, where x enters as FP16 and nothing here is lost
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,n,k", [(1, 8224, 8224), (5, 2464, 28768), (16, 8224, 8224), (32, 8224, 8224),
                                        (3, 96, 1056), (20, 96, 1056)])
def test_low_digits_of_a_linear(fmt, tokens, n, k):
    rng = np.random.default_rng(621)
    x, _ = low_linear(rng, tokens, k, 1, fmt)
    b = d.block(fmt)
    at = rng.integers(0, k // b, n) * b + rng.integers(1, b, n)
    code = rng.choice([2, 10, 3, 5], n).astype(np.uint8)  # 1, -1, 1.5, 3
    value = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])[code & 7] * np.where(code & 8, -1.0, 1.0)
    codes = np.zeros((n, k // 2), np.uint8)
    codes[np.arange(n), at // 2] = code << (4 * (at % 2)).astype(np.uint8)
    scales = np.full((n, k // b), 0x38 if fmt == NV else 127, np.uint8)
    ts = torch.ones(1, dtype=torch.float32, device="cuda") if fmt == NV else None
    y = guarded(tokens * n, torch.float32, float("nan"))
    need = mx.mx_linear_workspace_bytes(tokens, k, n, fmt)
    assert (need > 0) == (k > 2000)
    mx.mx_linear_bf16(dev_bf16(synth.f32_to_bf16_bits(x.astype(np.float32))), tokens, k, k, fmt, dev_u8(codes),
                      dev_u8(oracle.scale_tile(scales)), ts, n, y, n, mx.MX_OUT_FP32)
    torch.cuda.synchronize()
    check_guards(y, what="linear")
    ref = x[:, at] * value
    tol = 1e-5 * np.abs(ref)
    if need:
        tops = np.abs(x).reshape(tokens, -1, b).max(2)[:, at // b]
        tol += 2.0 ** -22 * tops * np.abs(value)
        if fmt == NV:
            tol += 2.0 ** -39 * np.abs(x).max(1)[:, None] * np.abs(value)
    assert_close(y.view(tokens, n).double().cpu().numpy(), ref, tol, "low digits")
