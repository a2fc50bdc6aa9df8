"""GPU parity of mx_linear_bf16 where it takes a workspace (weights of many bytes)
against the formula in binary64, on a sample of the rows.

Tolerance, FP32 out: E = 1e-5 sum_k |x||w| (the accumulation bound of the GEMM tests)
+ 2^-22 sum over blocks (32 of K for MXFP4, 16 for NVFP4) of (max |x| of the block)
(sum |w|) (what eight FP4 digits lose of an element far below its block's largest; the
sizes without a workspace lose less)
+ 2^-39 (max |x| of the token) (sum |w|) (NVFP4: the least E4M3 scale).  BF16 out:
plus one BF16 ulp.  With an epilogue as in the tests of the smaller sizes.
"""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
import oracle
from block_scaled_fp4_bf16_gb300 import synth
from tests.gpu_helpers import bf16_bits_to_f64, check_guards, dev_bf16, dev_u8, guarded
from tests.test_gpu_few_tokens import FMTS, MX, NV, assert_close, block, gelu, strided, ulp, x_bits

pytestmark = pytest.mark.gpu


class Wide:
    """A weight on the device, and the binary64 values of some of its rows."""

    def __init__(self, n, k, fmt, seed, lo=None, hi=None):
        lo, hi = (lo, hi) if lo is not None else ((116, 124) if fmt == MX else (0x20, 0x48))
        self.n, self.k, self.fmt = n, k, fmt
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
        self.s = np.random.default_rng(seed).integers(lo, hi + 1, (n, k // block(fmt)), dtype=np.uint8)
        self.scales = dev_u8(oracle.scale_tile(self.s))
        self.ts = None if fmt == MX else torch.full((1,), 0.03, dtype=torch.float32, device="cuda")
        rng = np.random.default_rng(seed + 1)
        self.rows = np.unique(np.r_[0:min(n, 33), n - min(n, 33):n, rng.integers(0, n, 150)])

    def value(self):
        dec = oracle.ue8m0_decode if self.fmt == MX else oracle.e4m3_decode
        table = np.array([dec(b) for b in range(256)])
        codes = self.codes[torch.from_numpy(self.rows).cuda()].cpu().numpy()
        v = oracle.e2m1_decode_array(codes, self.k).reshape(len(self.rows), -1, block(self.fmt))
        v = (v * table[self.s[self.rows]][:, :, None]).reshape(len(self.rows), self.k)
        return v if self.ts is None else v * float(self.ts.item())


def run(bits, w, out_fp32=True, ld_x=None, ld_y=None, bias=None, beta=0.0, gelu_on=False, y_in=None):
    t, k = bits.shape
    ld_x, ld_y = ld_x or k, ld_y or w.n
    body = guarded(t * ld_y, torch.float32 if out_fp32 else torch.bfloat16, float("nan"))
    y = body.view(t, ld_y)
    y._mx_guard = body._mx_guard
    if y_in is not None:
        y[:, :w.n] = y_in
    need = mx.mx_linear_workspace_bytes(t, k, w.n, w.fmt)
    ws = guarded(max(need, 1), torch.uint8, 0xA5)  # (unused where need is 0)
    mx.mx_linear_bf16(strided(bits, ld_x), t, k, ld_x, w.fmt, w.codes, w.scales, w.ts, w.n, y, ld_y,
                      mx.MX_OUT_FP32 if out_fp32 else mx.MX_OUT_BF16, bias, beta, gelu_on, workspace=ws)
    torch.cuda.synchronize()
    check_guards(y, ws, what="linear")
    if ld_y > w.n:
        assert torch.isnan(y[:, w.n:].float()).all(), "wrote past a row's end"
    return y[:, :w.n].float()


def pick(y, w):
    return y[:, torch.from_numpy(w.rows).cuda()].cpu().numpy().astype(np.float64)


def reference(bits, w):
    x, v = bf16_bits_to_f64(bits), w.value()
    a = np.abs(v)
    tol = 1e-5 * (np.abs(x) @ a.T)
    b = block(w.fmt)
    tol += 2.0 ** -22 * (np.abs(x).reshape(len(x), -1, b).max(2) @ a.reshape(len(a), -1, b).sum(2).T)
    if w.fmt == NV:
        tol += 2.0 ** -39 * np.abs(x).max(1)[:, None] * a.sum(1)[None]
    return x @ v.T, tol


# with a workspace (the first nine), and without it
SIZES = [(1, 8224, 8224), (4, 2464, 28768), (5, 75808, 1056), (8, 2424832 + 32, 32), (9, 2496, 31520),
         (16, 12320, 4128), (17, 1056, 27872), (31, 8224, 3616), (32, 96, 309600),
         (4, 2336, 28768), (5, 65568, 1056), (8, 2097152 + 32, 32), (9, 1600, 31520), (13, 1312, 25408),
         (32, 96, 16384), (7, 32, 12320)]


def test_which_sizes_take_a_workspace():
    assert all(mx.mx_linear_workspace_bytes(t, k, n, fmt) > 0 for t, n, k in SIZES[:9] for fmt in FMTS)
    assert all(mx.mx_linear_workspace_bytes(t, k, n, fmt) == 0 for t, n, k in SIZES[9:] for fmt in FMTS)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,n,k", SIZES)
def test_sizes(fmt, tokens, n, k):
    w, bits = Wide(n, k, fmt, 201), x_bits(tokens, k, 202)
    ref, tol = reference(bits, w)
    got = run(bits, w)
    assert_close(pick(got, w), ref, tol, "fp32")
    assert torch.isfinite(got).all()
    assert_close(pick(run(bits, w, out_fp32=False), w), ref, tol + ulp(ref), "bf16")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("beta,bias,gelu_on", [(0.0, True, True), (-0.5, True, False)])
@pytest.mark.parametrize("tokens,n,k", [(3, 8224, 8224), (18, 2080, 14176)])
def test_epilogue_and_strides(fmt, beta, bias, gelu_on, tokens, n, k):
    w, bits = Wide(n, k, fmt, 211), x_bits(tokens, k, 212)
    rng = np.random.default_rng(213)
    b = rng.standard_normal(n).astype(np.float32)
    y_in = bf16_bits_to_f64(synth.f32_to_bf16_bits(rng.standard_normal((tokens, n)).astype(np.float32)))
    acc, e = reference(bits, w)
    yr, br = y_in[:, w.rows], b[w.rows]
    pre = acc + beta * yr + (br if bias else 0.0)
    ref = gelu(pre) if gelu_on else pre
    steps = 2.0 ** -22 * (np.abs(acc) + np.abs(beta * yr) + (np.abs(br) if bias else 0) + np.abs(ref))
    tol = 1.13 * (e + steps) + 44 * 2.0 ** -24 * np.abs(ref)
    got = run(bits, w, True, k + 24, n + 13, torch.from_numpy(b).cuda() if bias else None, beta, gelu_on,
              torch.from_numpy(y_in.astype(np.float32)).cuda() if beta else None)
    assert_close(pick(got, w), ref, tol, "epilogue")


@pytest.mark.parametrize("fmt", FMTS)
def test_wide_ranges(fmt):
    """Activations whose blocks differ by many binades, weights over the scales' whole range."""
    t, n, k = 20, 4128, 8192
    w = Wide(n, k, fmt, 221, *((64, 190) if fmt == MX else (0, 0x7E)))
    x = bf16_bits_to_f64(x_bits(t, k, 222))
    x *= 2.0 ** np.tile(np.arange(-28, 28, 7), k // 256).repeat(32)[None, :]
    x[1] *= 2.0 ** -60
    x[2, ::3] = 0.0
    x[3] = 0.0
    x[4, 128:] *= 2.0 ** np.random.default_rng(1).integers(-20, 1, k - 128)
    bits = synth.f32_to_bf16_bits(x.astype(np.float32))
    ref, tol = reference(bits, w)
    got = run(bits, w)
    assert_close(pick(got, w), ref, tol, "ranges")
    assert (got[3] == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_nonfinite_activations_stay_in_their_token(fmt):
    t, n, k = 18, 4128, 8160
    w, bits = Wide(n, k, fmt, 231), x_bits(t, k, 232)
    clean = run(bits, w)
    bad = bits.copy()
    bad[2, 5], bad[4, 4000], bad[17, k - 1] = 0x7FC0, 0x7F80, 0xFF80
    got = run(bad, w)
    v, some = w.value(), pick(got, w)
    for r in range(t):
        if r == 2:
            assert torch.isnan(got[r]).all()
        elif r in (4, 17):
            col, sign = (4000, 1) if r == 4 else (k - 1, -1)
            nz = v[:, col] != 0
            assert not torch.isfinite(got[r]).any()
            assert (some[r][nz] == sign * np.sign(v[nz, col]) * np.inf).all() and np.isnan(some[r][~nz]).all()
        else:
            assert (got[r] == clean[r]).all()


def test_nan_scales():
    """UE8M0 bytes 255 (NaN) in one block of two rows, one of them with an infinite x there."""
    n, k = 8224, 8224
    w, bits = Wide(n, k, MX, 241, 127, 127), x_bits(2, k, 242)
    s = w.s.copy()
    s[130, 200], s[n - 1, 0] = 255, 255
    w.scales = dev_u8(oracle.scale_tile(s))
    bits[1, 32 * 200] = 0x7F80
    got = run(bits, w).isnan().cpu()
    bad = torch.zeros(n, dtype=torch.bool)
    bad[130] = bad[n - 1] = True
    assert torch.equal(got[0], bad)
    assert got[1][bad].all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,n,k", [(2, 8192, 8192), (32, 96, 309600)])
def test_bits_do_not_depend_on_the_order_of_arrival(fmt, tokens, n, k):
    w, bits = Wide(n, k, fmt, 251), x_bits(tokens, k, 252)
    first = run(bits, w)
    for _ in range(10):
        assert torch.equal(run(bits, w), first)


def test_streams_and_graph():
    """Calls in a captured graph and on two streams at once, each with its own workspace."""
    t, n, k = 4, 8224, 8224
    w = Wide(n, k, NV, 261)
    xs = [dev_bf16(x_bits(t, k, 262 + i)) for i in range(4)]
    call = lambda x, y: mx.mx_linear_bf16(x, t, k, k, NV, w.codes, w.scales, w.ts, n, y, n, mx.MX_OUT_FP32)
    want = [torch.empty(t, n, dtype=torch.float32, device="cuda") for _ in xs]
    for x, y in zip(xs, want):
        call(x, y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [torch.empty_like(y) for y in want]
    for rep in range(3):
        for i, (x, y) in enumerate(zip(xs, got)):
            with torch.cuda.stream(streams[i % 2]):
                call(x, y)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    got = [torch.zeros_like(y) for y in want]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for x, y in zip(xs, got):
            call(x, y)
    for _ in range(3):
        for y in got:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    # by addresses, on a given stream: without a workspace, by the other kernel
    y = torch.zeros_like(want[0])
    mx.mx_linear_bf16(xs[0].data_ptr(), t, k, k, NV, w.codes, w.scales, w.ts, n, y, n, mx.MX_OUT_FP32,
                      stream=streams[0])
    torch.cuda.synchronize()
    assert torch.allclose(y, want[0], rtol=1e-4, atol=1e-3)


def test_workspace_sizes():
    assert mx.mx_linear_workspace_bytes(1, 4096, 4096, MX) == 0
    assert mx.mx_linear_workspace_bytes(1, 8192, 28672, MX) > 0
    assert mx.mx_linear_workspace_bytes(33, 8192, 28672, MX) == 0
    assert mx.mx_linear_workspace_bytes(1, 8200, 28672, MX) == 0
    assert mx.mx_linear_workspace_bytes(1, 8192, 28672, 7) == 0
