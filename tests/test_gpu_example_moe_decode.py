"""The decoding example: its graph gives the tokens of plain calls, and its logits are
those of the formulas in binary64 (with the choice of experts that it made)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
import oracle

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_decode.py")


def example():
    spec = importlib.util.spec_from_file_location("moe_decode", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", [mx.MX_FMT_MXFP4, mx.MX_FMT_NVFP4])
@pytest.mark.parametrize("tokens", [1, 5])
def test_graph_gives_the_tokens_of_plain_calls(fmt, tokens):
    ex = example()
    d = ex.Decoder(ex.Model(2, 256, 128, 8, 2, 512, fmt), tokens)
    first = torch.arange(tokens, device="cuda") * 3
    out = d.decode(first, 6)
    d.ids.copy_(first)
    for i in range(6):
        d.step()
        assert torch.equal(d.ids, out[i])
    assert (out >= 0).all() and (out < 512).all()


def unpack(weights, fmt, rows, k):
    """The binary64 values that (codes, scales, tensor scale) stand for, [count, rows, k]."""
    codes, scales, ts = weights
    block = 32 if fmt == mx.MX_FMT_MXFP4 else 16
    dec = oracle.ue8m0_decode if fmt == mx.MX_FMT_MXFP4 else oracle.e4m3_decode
    table = np.array([dec(b) for b in range(256)])
    out = []
    for e in range(codes.shape[0]):
        r, c = np.meshgrid(np.arange(rows), np.arange(k // block), indexing="ij")
        tiles = (k // block + 3) // 4
        at = ((r // 128) * tiles + c // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4
        s = table[scales[e].cpu().numpy()[at]] * (1.0 if ts is None else float(ts[e].item()))
        v = oracle.e2m1_decode_array(codes[e].cpu().numpy(), k).reshape(rows, -1, block)
        out.append((v * s[:, :, None]).reshape(rows, k))
    return np.stack(out)


@pytest.mark.parametrize("fmt", [mx.MX_FMT_MXFP4, mx.MX_FMT_NVFP4])
def test_logits(fmt):
    ex = example()
    tokens, hidden, inter, experts, vocab = 3, 256, 128, 8, 512
    model = ex.Model(1, hidden, inter, experts, 2, vocab, fmt)
    d = ex.Decoder(model, tokens)
    d.ids.copy_(torch.tensor([3, 100, 511], device="cuda"))
    x = model.embedding[d.ids]
    d.step()
    xn = model.norm(x).double().cpu().numpy()
    _, moe = model.layers[0]
    gate, up, down = (unpack(w, fmt, r, k) for w, r, k in zip(moe.tensors, (inter, inter, hidden),
                                                              (hidden, hidden, inter)))
    ids, w = d.choice.cpu().numpy(), d.weights.double().cpu().numpy()
    y = np.zeros((tokens, hidden))
    for t in range(tokens):
        for j in range(2):
            g, u = gate[ids[t, j]] @ xn[t], up[ids[t, j]] @ xn[t]
            y[t] += w[t, j] * (down[ids[t, j]] @ (g / (1 + np.exp(-g)) * u))
    # y, x + y and its norm are BF16: one rounding each of what they have, 2^-8
    got = d.y.double().cpu().numpy()
    assert (np.abs(got - y) <= 2.0 ** -8 * np.abs(y) + 1e-4 * np.abs(y).max()).all()
    last = model.norm(x + d.y).double().cpu().numpy()
    head = unpack(model.head, fmt, vocab, hidden)[0]
    tol = 1e-5 * (np.abs(last) @ np.abs(head).T)
    assert (np.abs(d.logits.double().cpu().numpy() - last @ head.T) <= tol).all()
