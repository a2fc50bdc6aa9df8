"""The mixture of experts where its kernels change their way: one to four tokens (the
digits of x by token, made by the launch before), groups around the size up to which two
stages of the down product share a slot, odd numbers of stages, infinities and NaN.

References and tolerances are those of the other few-token tests.
"""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from block_scaled_fp4_bf16_gb300 import synth
from tests.gpu_helpers import bf16_bits_to_f64, check_guards, dev_bf16, guarded
from tests.test_gpu_few_tokens import FMTS, Layer, assert_close, choice, run_experts, run_route, x_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("hidden,inter,experts,top_k", [(32, 64, 4, 2), (4128, 96, 3, 2), (8224, 32, 2, 1)])
def test_layer_of_one_to_five_tokens(fmt, tokens, hidden, inter, experts, top_k):
    """The layer against binary64 with the choice that it made, and bit for bit its parts."""
    layer = Layer(experts, hidden, inter, fmt, mx.MX_ACT_SILU, 801)
    bits = x_bits(tokens, hidden, 802)
    rb = synth.bf16_normal(experts, hidden, 1.5 * hidden ** -0.5, 803)
    ids, w = run_route(bits, rb, None, top_k, 1)
    ref, tol = layer.ref(bf16_bits_to_f64(bits), ids, w)
    want = run_experts(layer, bits, ids, w, ld_x=hidden + 8)
    assert_close(want, ref, tol, "experts")
    ws = guarded(mx.mx_moe_workspace_bytes(tokens, hidden, inter, top_k), torch.uint8, 0xFF)
    gi, gw = guarded(tokens * top_k, torch.int32, 5), guarded(tokens * top_k, torch.float32, 0.5)
    y = guarded(tokens * hidden, torch.bfloat16, float("nan"))
    mx.mx_moe_layer_bf16(dev_bf16(bits), tokens, hidden, dev_bf16(rb), None, top_k, True, layer.moe, gi, gw, y,
                         hidden, ws)
    torch.cuda.synchronize()
    check_guards(ws, gi, gw, y, what="layer")
    assert (gi.view(tokens, top_k).cpu().numpy() == ids).all()
    assert (y.view(tokens, hidden).float().cpu().numpy().astype(np.float64) == want).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("inter", [32, 288, 544, 1312])
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 6, 7, 8, 9, 15, 16, 17, 40])
def test_experts_crowded_into_groups_of_every_size(fmt, inter, tokens):
    """Every token to expert 1; and every third to expert 0 instead."""
    layer = Layer(2, 96, inter, fmt, mx.MX_ACT_GELU, 811)
    bits = x_bits(tokens, 96, 812)
    w = np.random.default_rng(813).random((tokens, 1)).astype(np.float32)
    for ids in (np.ones((tokens, 1), np.int32), (np.arange(tokens) % 3 != 0).astype(np.int32)[:, None]):
        ref, tol = layer.ref(bf16_bits_to_f64(bits), ids, w)
        assert_close(run_experts(layer, bits, ids, w), ref, tol, "crowded")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [3, 4, 12])
def test_nonfinite_tokens_leave_the_others_alone(fmt, tokens):
    """All tokens share the experts, so their digits stand side by side in a product."""
    layer = Layer(2, 416, 160, fmt, mx.MX_ACT_SILU, 821)
    bits = x_bits(tokens, 416, 822)
    ids, w = choice(tokens, 2, 2, 823)
    clean = run_experts(layer, bits, ids, w)
    bad = bits.copy()
    bad[0, 415], bad[2, 7] = 0x7F80, 0x7FC0
    got = run_experts(layer, bad, ids, w)
    assert np.isnan(got[[0, 2]]).all()
    keep = [t for t in range(tokens) if t not in (0, 2)]
    assert (got[keep] == clean[keep]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_one_token_many_calls_give_the_same_bits(fmt):
    layer = Layer(8, 1056, 544, fmt, mx.MX_ACT_SILU, 831)
    for tokens in (1, 4):
        bits = x_bits(tokens, 1056, 832)
        ids, w = choice(tokens, 8, 3, 833)
        first = run_experts(layer, bits, ids, w)
        for _ in range(10):
            assert (run_experts(layer, bits, ids, w) == first).all()
