"""The decoding example for as many sequences as its layers take (64): more than one call of
the output projection takes."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests.test_gpu_example_moe_decode import example, unpack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [mx.MX_FMT_MXFP4, mx.MX_FMT_NVFP4])
@pytest.mark.parametrize("tokens", [32, 33, 64])
def test_steps_and_logits(fmt, tokens):
    ex = example()
    hidden, vocab = 256, 512
    model = ex.Model(1, hidden, 128, 8, 2, vocab, fmt)
    d = ex.Decoder(model, tokens)
    first = torch.arange(tokens, device="cuda") * 7
    out = d.decode(first, 3)
    d.ids.copy_(first)
    for i in range(3):
        d.step()
        assert torch.equal(d.ids, out[i])
    d.ids.copy_(first)
    d.step()
    last = model.norm(model.embedding[first] + d.y).double().cpu().numpy()
    head = unpack(model.head, fmt, vocab, hidden)[0]
    tol = 1e-5 * (np.abs(last) @ np.abs(head).T)
    assert (np.abs(d.logits.double().cpu().numpy() - last @ head.T) <= tol).all()
