"""The decoding step's calls together, as a decoder makes them: rotate, store, attend and sample, step
after step on one growing cache, eagerly, captured, and on two streams at once."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests import decode_ref as ref
from tests.gpu_helpers import check_guards, guarded

pytestmark = pytest.mark.gpu


class Decoder:
    """Queries, keys and values come in one row of a projection; logits are given."""

    def __init__(self, sequences=5, q_heads=6, kv_heads=2, dim=64, n=1, context=160, vocab=5003, seed=0):
        self.b, self.qh, self.kh, self.d, self.n, self.v = sequences, q_heads, kv_heads, dim, n, vocab
        g = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.rand = rand
        self.w = [(1 + 0.2 * rand(dim)).to(torch.bfloat16) for _ in range(2)]
        self.f = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float32, device="cuda") / dim)
        self.norm = mx.qk_norm(q_heads, kv_heads, dim, *self.w, self.f)
        per = -(-context // 32)
        pages = sequences * per
        self.table = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).view(sequences, per)
        self.codes = [guarded(pages * kv_heads * 32 * dim, fill=0x7F) for _ in range(2)]
        self.scales = [guarded(pages * kv_heads, fill=0xFF) for _ in range(2)]
        self.cache = mx.kv_cache(self.codes[0], self.scales[0], self.codes[1], self.scales[1], pages, 32, kv_heads, dim)
        self.pages = pages
        rows = sequences * n
        self.ld = (q_heads + 2 * kv_heads) * dim
        self.x = torch.empty(rows, self.ld, dtype=torch.bfloat16, device="cuda")
        self.qkv = torch.empty_like(self.x)
        self.logits = torch.empty(sequences, vocab, device="cuda")
        self.u = torch.empty(sequences, device="cuda")
        self.lengths = torch.zeros(sequences, dtype=torch.int32, device="cuda")
        self.positions = torch.empty(rows, dtype=torch.int32, device="cuda")
        self.out = torch.empty(rows, q_heads * dim, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty(rows, q_heads, device="cuda")
        self.ids = torch.empty(sequences, dtype=torch.int32, device="cuda")
        self.ws = guarded(mx.mx_attention_workspace_bytes(sequences, n, q_heads, self.cache))
        self.t = torch.full((sequences,), 0.8, device="cuda")
        self.k = torch.full((sequences,), 40, dtype=torch.int32, device="cuda")
        self.p = torch.full((sequences,), 0.9, device="cuda")

    def inputs(self):
        self.x.copy_(self.rand(*self.x.shape).to(torch.bfloat16))
        self.logits.copy_(2 * self.rand(*self.logits.shape))
        self.u.copy_(torch.rand(self.b, device="cuda"))

    def step(self):
        t, ld, at = self.b * self.n, self.ld, self.qh * self.d
        self.lengths += self.n
        self.positions.copy_((self.lengths[:, None] - self.n + torch.arange(self.n, device="cuda", dtype=torch.int32)).view(-1))
        self.qkv.copy_(self.x)
        k, v = self.qkv[:, at:], self.qkv[:, at + self.kh * self.d:]
        mx.mx_qk_norm_rope_bf16(self.qkv, ld, k, ld, t, self.positions, self.norm, self.qkv, ld, k, ld)
        mx.mx_kv_append_bf16(k, ld, v, ld, t, None, self.table, self.table.shape[1], self.lengths, self.b, self.cache)
        mx.mx_attention_bf16(self.qkv, ld, self.qh, self.b, self.n, self.table, self.table.shape[1], self.lengths, self.cache,
                             self.d ** -0.5, 0, self.out, at, self.lse, self.ws)
        mx.mx_sample(self.logits, self.b, self.v, self.v, mx.MX_OUT_FP32, self.t, self.k, self.p, None, self.u, self.ids)

    def results(self):
        return [x.clone() for x in (self.qkv, *self.codes, *self.scales, self.out, self.lse, self.ids)]


@pytest.mark.parametrize("n", [1, 3])
def test_steps_against_the_definitions(n):
    d = Decoder(n=n)
    cache = ref.Cache(d.pages, 32, d.kh, d.d, d.table.cpu().numpy())
    cache.codes = [np.full_like(c, 0x7F) for c in cache.codes]
    cache.scales = [np.full_like(s, 0xFF) for s in cache.scales]
    f64 = lambda x: x.double().cpu().numpy()  # noqa: E731
    for step in range(40):
        d.inputs()
        d.step()
        check_guards(*d.codes, *d.scales, d.ws)
        rows, lengths = d.b * n, d.lengths.cpu().numpy()
        qkv, x = f64(d.qkv).reshape(rows, -1, d.d), f64(d.x).reshape(rows, -1, d.d)
        for lo, hi, w in ((0, d.qh, d.w[0]), (d.qh, d.qh + d.kh, d.w[1])):
            want = ref.norm_rotate(x[:, lo:hi], f64(w), 1e-6, d.positions.cpu().numpy(), f64(d.f), d.d, False)
            size = ref.rotate_size(ref.norm_rotate(x[:, lo:hi], f64(w), 1e-6, d.positions.cpu().numpy(), f64(d.f), 0, False),
                                   d.d, False)
            assert (np.abs(qkv[:, lo:hi] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size).all()
        k, v = qkv[:, d.qh:d.qh + d.kh], qkv[:, d.qh + d.kh:]
        cache.append((k, v), [n] * d.b, lengths)
        for which in range(2):
            assert np.array_equal(d.codes[which].cpu().numpy(), cache.codes[which].reshape(-1))
            assert np.array_equal(d.scales[which].cpu().numpy(), cache.scales[which].reshape(-1))
        if step % 8 == 7:
            out, lse, e_out, e_lse = ref.attention(cache, qkv[:, :d.qh], lengths, n, d.qh, np.float32(d.d ** -0.5), 0)
            assert (np.abs(f64(d.out).reshape(out.shape) - out) <= 2.0 ** -8 * np.abs(out) + e_out).all()
            assert (np.abs(f64(d.lse) - lse) <= e_lse).all()
        for b in range(d.b):
            want, _, near = ref.sample(f64(d.logits)[b], d.t[b].item(), 40, d.p[b].item(), 0.0, d.u[b].item())
            assert near > 2.0 ** -38 and int(d.ids[b]) == want
    assert mx.mx_device_status() == 0


def test_a_captured_step_gives_the_bits_of_eager_ones():
    eager, captured = Decoder(seed=3), Decoder(seed=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    captured.inputs()
    with torch.cuda.stream(side):
        captured.step()
    torch.cuda.current_stream().wait_stream(side)
    captured.lengths.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    captured.lengths.zero_()
    for c in (*captured.codes, *captured.scales):
        c.fill_(0x55)
    for c in (*eager.codes, *eager.scales):
        c.fill_(0x55)
    for _ in range(70):
        eager.inputs()
        for x in ("x", "logits", "u"):
            getattr(captured, x).copy_(getattr(eager, x))
        eager.step()
        graph.replay()
        for a, b in zip(eager.results(), captured.results()):
            assert torch.equal(a, b)
    assert mx.mx_device_status() == 0


def test_two_graphs_may_share_a_workspace_one_after_the_other():
    one, two = Decoder(seed=4, sequences=7), Decoder(seed=5, sequences=3, dim=128)
    want = []
    for d in (one, two):
        d.inputs()
        d.step()
        want.append(d.results())
        d.lengths.zero_()
    ws = one.ws if one.ws.numel() > two.ws.numel() else two.ws
    graphs = []
    for d in (one, two):
        d.ws = ws
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            d.step()
        graphs.append(graph)
    for _ in range(5):
        for d, graph, w in zip((one, two), graphs, want):
            d.lengths.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(d.results(), w))


def test_two_streams():
    ds = [Decoder(seed=6 + s, sequences=40, context=64) for s in range(2)]
    want = []
    for d in ds:
        d.inputs()
        for _ in range(30):
            d.step()
        want.append(d.results())
        d.lengths.zero_()
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(30):
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                d.step()
    torch.cuda.synchronize()
    for d, w in zip(ds, want):
        assert all(torch.equal(a, b) for a, b in zip(d.results(), w))
    assert mx.mx_device_status() == 0


def test_a_given_stream():
    d = Decoder(seed=9)
    d.inputs()
    d.step()
    want = d.results()
    d.lengths.zero_()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    t, ld, at = d.b, d.ld, d.qh * d.d
    d.lengths += 1
    d.qkv.copy_(d.x)
    torch.cuda.synchronize()
    k, v = d.qkv[:, at:], d.qkv[:, at + d.kh * d.d:]
    for stream in (s, s.cuda_stream):
        d.qkv.copy_(d.x)
        torch.cuda.synchronize()
        mx.mx_qk_norm_rope_bf16(d.qkv, ld, k, ld, t, d.positions, d.norm, d.qkv, ld, k, ld, stream=stream)
        mx.mx_kv_append_bf16(k, ld, v, ld, t, None, d.table, d.table.shape[1], d.lengths, d.b, d.cache, stream=stream)
        mx.mx_attention_bf16(d.qkv, ld, d.qh, d.b, 1, d.table, d.table.shape[1], d.lengths, d.cache, d.d ** -0.5, 0, d.out, at,
                             d.lse, d.ws, stream=stream)
        mx.mx_sample(d.logits, d.b, d.v, d.v, mx.MX_OUT_FP32, d.t, d.k, d.p, None, d.u, d.ids, stream=stream)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(d.results(), want))


def test_forward_and_gradients_captured():
    t, q, k, dim = 50, 6, 2, 64
    g = torch.Generator("cuda").manual_seed(1)
    x, dy = ((torch.randn(t, (q + k) * dim, device="cuda", generator=g)).to(torch.bfloat16) for _ in range(2))
    w = [(1 + 0.1 * torch.randn(dim, device="cuda", generator=g)).to(torch.bfloat16) for _ in range(2)]
    f = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float32, device="cuda") / dim)
    norm, pos, ld, at = mx.qk_norm(q, k, dim, *w, f), torch.arange(t, dtype=torch.int32, device="cuda"), (q + k) * dim, q * dim
    ws = torch.empty(mx.mx_qk_norm_rope_backward_workspace_bytes(t, norm), dtype=torch.uint8, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw = [torch.empty(dim, device="cuda") for _ in range(2)]

    def both():
        mx.mx_qk_norm_rope_bf16(x, ld, x[:, at:], ld, t, pos, norm, y, ld, y[:, at:], ld)
        mx.mx_qk_norm_rope_backward_bf16(x, ld, x[:, at:], ld, dy, ld, dy[:, at:], ld, t, pos, norm, dx, ld, dx[:, at:], ld,
                                         *dw, ws)
    both()
    want = [v.clone() for v in (y, dx, *dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for v in (y, dx, *dw):
        v.zero_()
    ws.fill_(0xFF)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip((y, dx, *dw), want))
