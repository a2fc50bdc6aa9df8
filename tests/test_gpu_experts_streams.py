"""Calls of the experts and of the layer on two streams at once, each stream with a workspace
of its own, beside a linear on a third: the same bits as one after the other.  (The experts'
kernel is launched cooperatively: its CTAs are resident together or not yet at all.)"""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from block_scaled_fp4_bf16_gb300 import synth
from tests.gpu_helpers import dev_bf16
from tests.test_gpu_few_tokens import FMTS, Layer, Weight, choice, x_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [1, 8, 48])
def test_two_streams(fmt, tokens):
    h, i, e, k, calls = 1056, 544, 8, 3, 30
    layers = [Layer(e, h, i, fmt, mx.MX_ACT_SILU, 901 + 5000 * s) for s in range(2)]
    head = Weight(288, h, fmt, 902)
    codes, scales, ts = head.device()
    bits = [x_bits(tokens, h, 903 + s) for s in range(2)]
    xs = [dev_bf16(b) for b in bits]
    router = dev_bf16(synth.bf16_normal(e, h, 1.5 * h ** -0.5, 904))
    ids, w = choice(tokens, e, k, 905)
    ids, w = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    new = lambda *s, dtype=torch.bfloat16: torch.full(s, 7, dtype=dtype, device="cuda")  # noqa: E731
    ws = [new(mx.mx_moe_workspace_bytes(tokens, h, i, k), dtype=torch.uint8) for _ in range(2)]
    own = [(new(tokens, k, dtype=torch.int32), new(tokens, k, dtype=torch.float32)) for _ in range(2)]

    def step(s, y, z):
        mx.mx_moe_experts_bf16(xs[s], tokens, h, ids, w, k, layers[s].moe, y, h, ws[s])
        mx.mx_moe_layer_bf16(xs[s], tokens, h, router, None, k, True, layers[s].moe, *own[s], z, h, ws[s])

    def linear(y):
        rows = min(tokens, mx.MX_LINEAR_MAX_TOKENS)
        mx.mx_linear_bf16(xs[0], rows, h, h, fmt, codes, scales, ts, 288, y, 288, mx.MX_OUT_FP32)

    want = [(new(tokens, h), new(tokens, h)) for _ in range(2)]
    want_linear = new(tokens, 288, dtype=torch.float32)
    for s in range(2):
        step(s, *want[s])
    linear(want_linear)
    torch.cuda.synchronize()
    assert mx.mx_device_status() == mx.MX_OK
    got = [[(new(tokens, h), new(tokens, h)) for _ in range(calls)] for _ in range(2)]
    got_linear = [new(tokens, 288, dtype=torch.float32) for _ in range(calls)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for c in range(calls):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                step(s, *got[s][c])
        with torch.cuda.stream(streams[2]):
            linear(got_linear[c])
    torch.cuda.synchronize()
    assert mx.mx_device_status() == mx.MX_OK
    for s in range(2):
        assert torch.isfinite(want[s][0].float()).all() and torch.isfinite(want[s][1].float()).all()
        for y, z in got[s]:
            assert torch.equal(y, want[s][0]) and torch.equal(z, want[s][1])
    assert all(torch.equal(y, want_linear) for y in got_linear)
    assert np.isfinite(want_linear[:1].cpu().numpy()).all()
