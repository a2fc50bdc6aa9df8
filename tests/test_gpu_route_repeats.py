"""The router where its CTAs have next to nothing to do before they write to one another's
shared memory (hidden 32, a launch behind a launch): every one of many calls right."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from block_scaled_fp4_bf16_gb300 import synth
from tests.gpu_helpers import dev_bf16
from tests.test_gpu_few_tokens import route_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 16, 4), (8, 512, 16), (64, 512, 8)])
def test_many_short_calls(tokens, experts, top_k):
    """Logits are small integers: exact, with ties."""
    h, calls, rng = 32, 200, np.random.default_rng(11)
    x = rng.integers(-3, 4, (tokens, h)).astype(np.float32)
    r = rng.integers(-3, 4, (experts, h)).astype(np.float32)
    rid, rw, _ = route_ref(x.astype(np.float64), r.astype(np.float64), None, top_k, 1)
    xd, rd = dev_bf16(synth.f32_to_bf16_bits(x)), dev_bf16(synth.f32_to_bf16_bits(r))
    ids = torch.full((calls, tokens, top_k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((calls, tokens, top_k), float("nan"), device="cuda")
    torch.cuda.synchronize()
    for i in range(calls):
        mx.mx_moe_route_bf16(xd, tokens, h, h, rd, experts, None, top_k, True, ids[i], w[i])
    torch.cuda.synchronize()
    assert (ids.cpu().numpy() == rid[None]).all()
    assert (np.abs(w.cpu().numpy().astype(np.float64) - rw[None]) <= 2e-5 * rw[None]).all()
