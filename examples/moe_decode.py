"""Decoding with FP4 experts: a stack of mixture-of-experts layers and an FP4 output
projection, a few tokens a step, the whole step one CUDA graph.

    python examples/moe_decode.py [--tokens 8] [--format mxfp4] [--check]

The weights are random BF16 matrices, quantized once (mx_quantize_bf16).  A step takes
the token ids of the last one, looks up their embeddings, runs per layer
    x = x + moe(norm(x))        mx_moe_layer_bf16 (router, chosen experts, their sum)
and ends with the logits of the next tokens (mx_linear_bf16) and their largest.
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import block_scaled_fp4_bf16_gb300 as mx  # noqa: E402


def quantized(w, fmt):
    """(codes, scales, tensor scale) of a BF16 matrix, or of a stack of them."""
    stack = w if w.dim() == 3 else w[None]
    count, rows, k = stack.shape
    codes = torch.empty(count, rows, k // 2, dtype=torch.uint8, device=w.device)
    scales = torch.zeros(count, mx.mx_scale_bytes(rows, k, fmt, mx.MX_SCALE_TCGEN05), dtype=torch.uint8,
                         device=w.device)
    ts = torch.empty(count, dtype=torch.float32, device=w.device) if fmt == mx.MX_FMT_NVFP4 else None
    need = mx.mx_quantize_workspace_bytes(rows, k, fmt)
    ws = torch.empty(need, dtype=torch.uint8, device=w.device) if need else None
    for e in range(count):
        mx.mx_quantize_bf16(stack[e], rows, k, k, fmt, mx.MX_SCALE_TCGEN05, codes[e], scales[e],
                            None if ts is None else ts[e:e + 1], ws)
    return codes, scales, ts


class Model:
    """`layers` mixtures of experts over `hidden`, and the projection onto `vocab`."""

    def __init__(self, layers, hidden, inter, experts, top_k, vocab, fmt, seed=0):
        self.hidden, self.inter, self.experts, self.top_k = hidden, inter, experts, top_k
        self.vocab, self.fmt = vocab, fmt
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def matrix(*shape):
            w = torch.randn(*shape, device="cuda", generator=gen) * shape[-1] ** -0.5
            return w.to(torch.bfloat16)

        self.embedding = matrix(vocab, hidden) * hidden ** 0.5
        self.layers = []
        for _ in range(layers):
            plain = [matrix(experts, inter, hidden), matrix(experts, inter, hidden),
                     matrix(experts, hidden, inter)]
            moe = mx.moe_weights(fmt, experts, hidden, inter, *(quantized(w, fmt) for w in plain))
            self.layers.append((matrix(experts, hidden), moe))
        self.head = quantized(matrix(vocab, hidden), fmt)

    def norm(self, x):
        return torch.nn.functional.rms_norm(x, (self.hidden,))


class Decoder:
    """The step of `tokens` sequences as a CUDA graph."""

    def __init__(self, model, tokens):
        self.m, self.tokens = model, tokens
        new = lambda *s, dtype: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.ids = torch.zeros(tokens, dtype=torch.int64, device="cuda")
        self.y = new(tokens, model.hidden, dtype=torch.bfloat16)
        self.choice = new(tokens, model.top_k, dtype=torch.int32)
        self.weights = new(tokens, model.top_k, dtype=torch.float32)
        self.logits = new(tokens, model.vocab, dtype=torch.float32)
        self.moe_workspace = new(mx.mx_moe_workspace_bytes(tokens, model.hidden, model.inter, model.top_k),
                                 dtype=torch.uint8)
        # (the projection's calls take up to MX_LINEAR_MAX_TOKENS rows, one after the other)
        self.parts = [slice(i, min(i + mx.MX_LINEAR_MAX_TOKENS, tokens))
                      for i in range(0, tokens, mx.MX_LINEAR_MAX_TOKENS)]
        need = max(mx.mx_linear_workspace_bytes(p.stop - p.start, model.hidden, model.vocab, model.fmt)
                   for p in self.parts)
        self.head_workspace = new(need, dtype=torch.uint8) if need else None
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()  # builds what the first call builds, outside of the capture
        torch.cuda.current_stream().wait_stream(side)
        self.ids.zero_()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.step()
        self.ids.zero_()

    def step(self):
        m, t = self.m, self.tokens
        x = m.embedding[self.ids]
        for router, moe in m.layers:
            mx.mx_moe_layer_bf16(m.norm(x), t, m.hidden, router, None, m.top_k, True, moe, self.choice,
                                 self.weights, self.y, m.hidden, self.moe_workspace)
            x = x + self.y
        codes, scales, ts = m.head
        x = m.norm(x)
        for p in self.parts:
            mx.mx_linear_bf16(x[p], p.stop - p.start, m.hidden, m.hidden, m.fmt, codes, scales, ts, m.vocab,
                              self.logits[p], m.vocab, mx.MX_OUT_FP32, workspace=self.head_workspace)
        self.ids.copy_(self.logits.argmax(1))

    def decode(self, first, steps):
        """The next `steps` tokens of each sequence: [steps, tokens]."""
        self.ids.copy_(first)
        out = []
        for _ in range(steps):
            self.graph.replay()
            out.append(self.ids.clone())
        return torch.stack(out)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--format", choices=["mxfp4", "nvfp4"], default="mxfp4")
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--check", action="store_true", help="every step of the graph against plain calls")
    args = ap.parse_args()
    fmt = mx.MX_FMT_MXFP4 if args.format == "mxfp4" else mx.MX_FMT_NVFP4
    model = Model(args.layers, 2048, 1024, 64, 8, 32768, fmt)
    d = Decoder(model, args.tokens)
    first = torch.arange(args.tokens, device="cuda") * 7 % model.vocab
    out = d.decode(first, args.steps)
    mx.mx_device_status()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    d.decode(first, args.steps)
    torch.cuda.synchronize()
    dt = (time.perf_counter() - t0) / args.steps
    print(f"{args.tokens} sequences, {args.layers} layers of 64 experts ({args.format}): "
          f"{dt * 1e6:.0f} us a step, {args.tokens / dt:.0f} tokens/s")
    if args.check:
        d.ids.copy_(first)
        for i in range(args.steps):
            d.step()
            assert torch.equal(d.ids, out[i]), f"step {i} differs"
        print("the graph's tokens are those of the plain calls")


if __name__ == "__main__":
    main()
