"""The decoding example with attention and sampling: its graph gives the tokens of plain calls, and
its attention is that of the formulas in binary64 on the projections that it made."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests import decode_ref as ref
from tests.test_gpu_example_moe_decode import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 5, 40])
@pytest.mark.parametrize("attention,sampling", [((4, 2, 64), None), ((4, 2, 64), (0.8, 20, 0.9, 0.01)), (None, (1.0, 0, 1.0, 0.0)),
                                                ((2, 1, 128), (0.0, 0, 1.0, 0.0))])
def test_graph_gives_the_tokens_of_plain_calls(tokens, attention, sampling):
    ex = example()
    model = ex.Model(2, 256, 128, 8, 2, 512, mx.MX_FMT_MXFP4, attention=attention)
    d = ex.Decoder(model, tokens, sampling, context=64)
    first = torch.arange(tokens, device="cuda") * 3
    steps = 40
    u = torch.rand(steps, tokens, device="cuda", generator=torch.Generator("cuda").manual_seed(2)) if sampling else None
    out = d.decode(first, steps, u)
    d.restart()
    d.ids.copy_(first)
    for i in range(steps):
        if sampling:
            d.uniform.copy_(u[i])
        d.step()
        assert torch.equal(d.ids, out[i])
    assert (out >= 0).all() and (out < 512).all() and mx.mx_device_status() == 0
    if sampling and sampling[0] == 0.0:  # greedy is the largest logit
        assert torch.equal(d.ids, d.logits.argmax(1))


def test_no_more_steps_than_the_context():
    ex = example()
    d = ex.Decoder(ex.Model(1, 256, 128, 8, 2, 512, mx.MX_FMT_MXFP4, attention=(2, 1, 64)), 1, context=64)
    with pytest.raises(ValueError):
        d.decode(torch.zeros(1, dtype=torch.int64, device="cuda"), 65)


def test_attention_is_the_formulas():
    ex = example()
    tokens, q, kv, dim, hidden = 3, 4, 2, 64, 256
    model = ex.Model(1, hidden, 128, 8, 2, 512, mx.MX_FMT_MXFP4, attention=(q, kv, dim))
    d = ex.Decoder(model, tokens, context=64)
    a, c = model.attention[0], d.cache
    cache = ref.Cache(c.table.numel(), ex.PAGE, kv, dim, c.table.cpu().numpy())
    for which, x in enumerate(c.layers[0].tensors[::2]):
        x.fill_(0)
        cache.codes[which][:] = 0
    d.ids.copy_(torch.tensor([3, 100, 511], device="cuda"))
    f64 = lambda x: x.double().cpu().numpy()  # noqa: E731
    freq = f64(a.norm.tensors[2])
    for step in range(35):
        x = model.norm(model.embedding[d.ids])
        raw = torch.empty_like(c.qkv)
        d.linear(x, a.qkv, a.rows, raw, mx.MX_OUT_BF16)
        d.step()
        raw, qkv = (f64(v).reshape(tokens, -1, dim) for v in (raw, c.qkv))
        pos = np.full(tokens, step)
        rot = ref.norm_rotate(raw[:, :q + kv], np.ones(dim), 1e-6, pos, freq, dim, False)
        size = ref.rotate_size(ref.norm_rotate(raw[:, :q + kv], np.ones(dim), 1e-6, pos, freq, 0, False), dim, False)
        assert (np.abs(qkv[:, :q + kv] - rot) <= 2.0 ** -8 * np.abs(rot) + 2.0 ** -19 * size).all()
        cache.append((qkv[:, q:q + kv], raw[:, q + kv:]), [1] * tokens, [step + 1] * tokens)
    out, _, e_out, _ = ref.attention(cache, qkv[:, :q], [35] * tokens, 1, q, np.float32(dim ** -0.5), 0)
    assert (np.abs(f64(c.out).reshape(out.shape) - out) <= 2.0 ** -8 * np.abs(out) + e_out).all()
