"""Decoding with FP4 experts: a stack of mixture-of-experts layers and an FP4 output
projection, a few tokens a step, the whole step one CUDA graph.

    python examples/moe_decode.py [--tokens 8] [--format mxfp4] [--attention] [--sample] [--check]

The weights are random BF16 matrices, quantized once (mx_quantize_bf16).  A step takes
the token ids of the last one, looks up their embeddings, runs per layer
    x = x + attend(norm(x))     with --attention: mx_linear_bf16 (queries, keys, values),
                                mx_qk_norm_rope_bf16, mx_kv_append_bf16, mx_attention_bf16,
                                mx_linear_bf16
    x = x + moe(norm(x))        mx_moe_layer_bf16 (router, chosen experts, their sum)
and ends with the logits of the next tokens (mx_linear_bf16) and their largest, or with
--sample a draw from them (mx_sample).
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


class Attention:
    """A layer's attention: FP4 projections, norms of queries and keys, the rotation."""

    def __init__(self, matrix, hidden, q_heads, kv_heads, head_dim, fmt):
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.rows = (q_heads + 2 * kv_heads) * head_dim  # queries, keys, values
        self.qkv = quantized(matrix(self.rows, hidden), fmt)
        self.out = quantized(matrix(hidden, q_heads * head_dim), fmt)
        ones = torch.ones(head_dim, dtype=torch.bfloat16, device="cuda")
        inv_freq = 10000.0 ** (-torch.arange(0, head_dim, 2, dtype=torch.float32, device="cuda") / head_dim)
        self.norm = mx.qk_norm(q_heads, kv_heads, head_dim, ones, ones, inv_freq)


class Model:
    """`layers` mixtures of experts over `hidden`, and the projection onto `vocab`;
    attention: (q_heads, kv_heads, head_dim) of an attention before each mixture, or None."""

    def __init__(self, layers, hidden, inter, experts, top_k, vocab, fmt, seed=0, attention=None):
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
        self.attention = [Attention(matrix, hidden, *attention, fmt) for _ in self.layers] if attention else None

    def norm(self, x):
        return torch.nn.functional.rms_norm(x, (self.hidden,))


PAGE = 64  # tokens of a page of the cache


class Cache:
    """The sequences' keys and values, a pool of pages for each layer; one page table for all."""

    def __init__(self, model, tokens, context):
        per = -(-context // PAGE)
        new = lambda *s, dtype=torch.uint8: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.context = context
        self.table = torch.arange(tokens * per, dtype=torch.int32, device="cuda").view(tokens, per)
        self.lengths = torch.zeros(tokens, dtype=torch.int32, device="cuda")
        self.positions = new(tokens, dtype=torch.int32)
        self.layers = []
        for a in model.attention:
            codes = [new(tokens * per, a.kv_heads, PAGE, a.head_dim) for _ in range(2)]
            scales = [new(tokens * per, a.kv_heads, PAGE // mx.MX_CACHE_BLOCK) for _ in range(2)]
            self.layers.append(mx.kv_cache(codes[0], scales[0], codes[1], scales[1], tokens * per, PAGE, a.kv_heads,
                                           a.head_dim))
        a = model.attention[0]
        self.qkv = new(tokens, a.rows, dtype=torch.bfloat16)
        self.out = new(tokens, a.q_heads * a.head_dim, dtype=torch.bfloat16)
        self.projected = new(tokens, model.hidden, dtype=torch.bfloat16)
        self.workspace = new(mx.mx_attention_workspace_bytes(tokens, 1, a.q_heads, self.layers[0]))


class Decoder:
    """The step of `tokens` sequences as a CUDA graph.  sampling: (temperature, top_k, top_p, min_p),
    or None for the largest logit; context: most tokens of a sequence (with attention)."""

    def __init__(self, model, tokens, sampling=None, context=1024):
        self.m, self.tokens = model, tokens
        new = lambda *s, dtype: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.ids = torch.zeros(tokens, dtype=torch.int64, device="cuda")
        self.y = new(tokens, model.hidden, dtype=torch.bfloat16)
        self.choice = new(tokens, model.top_k, dtype=torch.int32)
        self.weights = new(tokens, model.top_k, dtype=torch.float32)
        self.logits = new(tokens, model.vocab, dtype=torch.float32)
        self.moe_workspace = new(mx.mx_moe_workspace_bytes(tokens, model.hidden, model.inter, model.top_k),
                                 dtype=torch.uint8)
        # (the projections' calls take up to MX_LINEAR_MAX_TOKENS rows, one after the other)
        self.parts = [slice(i, min(i + mx.MX_LINEAR_MAX_TOKENS, tokens))
                      for i in range(0, tokens, mx.MX_LINEAR_MAX_TOKENS)]
        shapes = [(model.hidden, model.vocab)]
        self.cache = Cache(model, tokens, context) if model.attention else None
        if self.cache:
            a = model.attention[0]
            shapes += [(model.hidden, a.rows), (a.q_heads * a.head_dim, model.hidden)]
        need = max(mx.mx_linear_workspace_bytes(p.stop - p.start, k, n, model.fmt)
                   for p in self.parts for k, n in shapes)
        self.linear_workspace = new(need, dtype=torch.uint8) if need else None
        if sampling is not None:
            kinds = (torch.float32, torch.int32, torch.float32, torch.float32)
            self.sampling = [torch.full((tokens,), v, dtype=t, device="cuda") for v, t in zip(sampling, kinds)]
            self.uniform = torch.zeros(tokens, device="cuda")
            self.sampled = new(tokens, dtype=torch.int32)
        else:
            self.sampling = None
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()  # builds what the first call builds, outside of the capture
        torch.cuda.current_stream().wait_stream(side)
        self.restart()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.step()
        self.restart()

    def restart(self):
        self.ids.zero_()
        if self.cache:
            self.cache.lengths.zero_()

    def linear(self, x, weight, rows, y, out_dtype):
        codes, scales, ts = weight
        k = x.shape[1]
        for p in self.parts:
            mx.mx_linear_bf16(x[p], p.stop - p.start, k, k, self.m.fmt, codes, scales, ts, rows, y[p], rows, out_dtype,
                              workspace=self.linear_workspace)

    def attend(self, x, a, cache):
        """The attention sublayer: x's queries over the cache and x's own keys and values."""
        c, t, ld, d = self.cache, self.tokens, a.rows, a.head_dim
        self.linear(x, a.qkv, ld, c.qkv, mx.MX_OUT_BF16)
        k, v = c.qkv[:, a.q_heads * d:], c.qkv[:, (a.q_heads + a.kv_heads) * d:]
        mx.mx_qk_norm_rope_bf16(c.qkv, ld, k, ld, t, c.positions, a.norm, c.qkv, ld, k, ld)  # in place
        mx.mx_kv_append_bf16(k, ld, v, ld, t, None, c.table, c.table.shape[1], c.lengths, t, cache)
        mx.mx_attention_bf16(c.qkv, ld, a.q_heads, t, 1, c.table, c.table.shape[1], c.lengths, cache, d ** -0.5, 0,
                             c.out, a.q_heads * d, None, c.workspace)
        self.linear(c.out, a.out, self.m.hidden, c.projected, mx.MX_OUT_BF16)
        return c.projected

    def step(self):
        m, t = self.m, self.tokens
        x = m.embedding[self.ids]
        if self.cache:
            self.cache.positions.copy_(self.cache.lengths)
            self.cache.lengths += 1
        for i, (router, moe) in enumerate(m.layers):
            if self.cache:
                x = x + self.attend(m.norm(x), m.attention[i], self.cache.layers[i])
            mx.mx_moe_layer_bf16(m.norm(x), t, m.hidden, router, None, m.top_k, True, moe, self.choice,
                                 self.weights, self.y, m.hidden, self.moe_workspace)
            x = x + self.y
        self.linear(m.norm(x), m.head, m.vocab, self.logits, mx.MX_OUT_FP32)
        if self.sampling is None:
            self.ids.copy_(self.logits.argmax(1))
        else:
            mx.mx_sample(self.logits, t, m.vocab, m.vocab, mx.MX_OUT_FP32, *self.sampling, self.uniform, self.sampled)
            self.ids.copy_(self.sampled)

    def decode(self, first, steps, uniform=None):
        """The next `steps` tokens of each sequence: [steps, tokens].  uniform: [steps, tokens] random
        numbers (with sampling)."""
        if self.cache and steps > self.cache.context:
            raise ValueError(f"{steps} steps of sequences of at most {self.cache.context} tokens")
        self.restart()
        self.ids.copy_(first)
        out = []
        for i in range(steps):
            if uniform is not None:
                self.uniform.copy_(uniform[i])
            self.graph.replay()
            out.append(self.ids.clone())
        return torch.stack(out)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--format", choices=["mxfp4", "nvfp4"], default="mxfp4")
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--attention", action="store_true", help="attention before each mixture of experts")
    ap.add_argument("--sample", action="store_true", help="draw the tokens (temperature 0.8, top-k 50, top-p 0.95)")
    ap.add_argument("--check", action="store_true", help="every step of the graph against plain calls")
    args = ap.parse_args()
    fmt = mx.MX_FMT_MXFP4 if args.format == "mxfp4" else mx.MX_FMT_NVFP4
    model = Model(args.layers, 2048, 1024, 64, 8, 32768, fmt, attention=(32, 8, 128) if args.attention else None)
    d = Decoder(model, args.tokens, (0.8, 50, 0.95, 0.0) if args.sample else None, max(args.steps, 64))
    first = torch.arange(args.tokens, device="cuda") * 7 % model.vocab
    gen = torch.Generator(device="cuda").manual_seed(1)
    uniform = torch.rand(args.steps, args.tokens, device="cuda", generator=gen) if args.sample else None
    out = d.decode(first, args.steps, uniform)
    mx.mx_device_status()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    d.decode(first, args.steps, uniform)
    torch.cuda.synchronize()
    dt = (time.perf_counter() - t0) / args.steps
    print(f"{args.tokens} sequences, {args.layers} layers of 64 experts ({args.format}): "
          f"{dt * 1e6:.0f} us a step, {args.tokens / dt:.0f} tokens/s")
    if args.check:
        d.restart()
        d.ids.copy_(first)
        for i in range(args.steps):
            if uniform is not None:
                d.uniform.copy_(uniform[i])
            d.step()
            assert torch.equal(d.ids, out[i]), f"step {i} differs"
        print("the graph's tokens are those of the plain calls")


if __name__ == "__main__":
    main()
