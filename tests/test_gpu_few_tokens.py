"""GPU parity of the few-token products (mx_linear_bf16, mx_moe_*) against the
formulas in binary64.

Tolerances, with S = sum_k |x||w|:

* linear, FP32 out: E = 1e-5 S + 2^-39 sum over groups of 128 of (max |x| of
  the group) (sum |w|); the first term is the accumulation bound of the GEMM
  tests, the second what FP16 can lose of an activation far below the largest
  of its 128 (nothing, when no element is below 2^-31 of it).  With an
  epilogue L (E + 2^-22 (|acc| + |beta y| + |bias| + |y|)) + 44 * 2^-24 |y|,
  L = 1.13 >= max |GELU'| (the GEMM epilogue's tolerance).
* BF16 out: the same plus one BF16 ulp.
* experts: the hidden value h = act(g) u carries dh = 1.13 E_g |u| + |act g| E_u
  + (E_g E_u) + 2^-20 |h| (silu and gelu have slope below 1.13), and enters the
  second product to within 2^-12 relative: z carries sum |w_d| (dh + 2^-12 |h|) +
  1e-5 sum |w_d||h| + the 2^-39 term; y the weighted sum of the z's, 2^-20 of
  their absolute sum, and one BF16 ulp.
* route: ids equal where the choice is exact or the gap to the next logit is
  above twice the logits' error; weights within 2e-5 relative.
"""
import math

import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
import oracle
from block_scaled_fp4_bf16_gb300 import synth
from tests.gpu_helpers import bf16_bits_to_f64, check_guards, dev_bf16, dev_u8, guarded

pytestmark = pytest.mark.gpu

MX, NV = mx.MX_FMT_MXFP4, mx.MX_FMT_NVFP4
TILED = mx.MX_SCALE_TCGEN05
FMTS = [MX, NV]


def block(fmt):
    return 32 if fmt == MX else 16


class Weight:
    """An FP4 matrix [rows, k]: random codes, scales of a spread, its fp64 values."""

    def __init__(self, rows, k, fmt, seed, lo=None, hi=None):
        lo, hi = (lo, hi) if lo is not None else ((116, 124) if fmt == MX else (0x20, 0x48))
        self.rows, self.k, self.fmt = rows, k, fmt
        self.codes = synth.fp4_codes(rows, k, seed)
        s = synth.scale_bytes(rows, k // block(fmt), lo, hi, seed + 1)
        self.scales = oracle.scale_tile(s)
        self.ts = None if fmt == MX else np.float32(0.01 * (1 + seed % 5))
        dec = oracle.ue8m0_decode if fmt == MX else oracle.e4m3_decode
        table = np.array([dec(b) for b in range(256)])
        v = oracle.e2m1_decode_array(self.codes, k)
        v = v.reshape(rows, -1, block(fmt)) * table[s][:, :, None]
        self.value = v.reshape(rows, k) * (1.0 if fmt == MX else float(self.ts))

    def device(self):
        ts = None if self.ts is None else torch.tensor([self.ts], dtype=torch.float32, device="cuda")
        return dev_u8(self.codes), dev_u8(self.scales), ts


class Stack:
    """`count` weights one after the other."""

    def __init__(self, count, rows, k, fmt, seed):
        self.w = [Weight(rows, k, fmt, seed + 7 * e) for e in range(count)]
        self.codes = dev_u8(np.stack([w.codes for w in self.w]))
        self.scales = dev_u8(np.stack([w.scales for w in self.w]))
        self.ts = None if fmt == MX else torch.tensor([w.ts for w in self.w], dtype=torch.float32,
                                                      device="cuda")
        self.device = (self.codes, self.scales, self.ts)


def x_bits(tokens, k, seed, sigma=1.0):
    return synth.bf16_normal(tokens, k, sigma, seed)


def strided(bits, ld, fill=0x7FC0):
    """Device BF16 [tokens, ld] whose columns past k hold NaN."""
    t, k = bits.shape
    full = np.full((t, ld), fill, dtype=np.uint16)
    full[:, :k] = bits
    return dev_bf16(full)


def fp16_loss(x, w):
    """2^-39 sum over 128-groups max|x| sum|w|: [tokens, rows]."""
    t, k = x.shape
    e = np.zeros((t, w.shape[0]))
    for g in range(0, k, 128):
        e += np.abs(x[:, g:g + 128]).max(1)[:, None] * np.abs(w[:, g:g + 128]).sum(1)[None]
    return 2.0 ** -39 * e


def ulp(v):
    a = np.maximum(np.abs(v), 2.0 ** -126)
    return 2.0 ** (np.floor(np.log2(a)) - 7)


def gelu(v):
    return 0.5 * v * np.array([math.erfc(-a / math.sqrt(2.0)) for a in v.ravel()]).reshape(v.shape)


def silu(v):
    return v / (1.0 + np.exp(-v))


def run_linear(bits, w, out_fp32=True, ld_x=None, ld_y=None, bias=None, beta=0.0, gelu_on=False,
               y_in=None, dev=None):
    t, k = bits.shape
    ld_x, ld_y = ld_x or k, ld_y or w.rows
    dt = torch.float32 if out_fp32 else torch.bfloat16
    body = guarded(t * ld_y, dt, float("nan"))
    y = body.view(t, ld_y)
    y._mx_guard = body._mx_guard
    if y_in is not None:
        y[:, :w.rows] = torch.from_numpy(y_in).cuda().to(dt)
    codes, scales, ts = dev or w.device()
    b = None if bias is None else torch.from_numpy(bias).cuda()
    mx.mx_linear_bf16(strided(bits, ld_x), t, k, ld_x, w.fmt, codes, scales, ts, w.rows, y, ld_y,
                      mx.MX_OUT_FP32 if out_fp32 else mx.MX_OUT_BF16, b, beta, gelu_on)
    torch.cuda.synchronize()
    check_guards(y, what="linear")
    if ld_y > w.rows:
        assert torch.isnan(y[:, w.rows:].float()).all(), "wrote past a row's end"
    return y[:, :w.rows].float().cpu().numpy().astype(np.float64)


def linear_ref(bits, w):
    x = bf16_bits_to_f64(bits)
    acc = x @ w.value.T
    return acc, 1e-5 * (np.abs(x) @ np.abs(w.value).T) + fp16_loss(x, w.value)


def assert_close(got, ref, tol, what):
    assert np.isfinite(got).all(), f"{what}: non-finite outputs"
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())}/{bad.size} outside; first at "
                           f"{np.argwhere(bad)[0]}: got {got[bad][0]!r} ref {ref[bad][0]!r} tol {tol[bad][0]!r}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 16, 17, 31, 32])
@pytest.mark.parametrize("n,k", [(32, 32), (96, 160), (160, 1056), (1056, 96)])
def test_linear_tokens(fmt, tokens, n, k):
    w, bits = Weight(n, k, fmt, 11), x_bits(tokens, k, 12)
    ref, tol = linear_ref(bits, w)
    assert_close(run_linear(bits, w), ref, tol, "fp32")
    assert_close(run_linear(bits, w, out_fp32=False), ref, tol + ulp(ref), "bf16")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,n,k", [(1, 2048, 4096), (3, 64, 28672), (8, 4096, 2048),
                                        (20, 512, 8192), (1, 9760, 64), (32, 1120, 3040)])
def test_linear_sizes(fmt, tokens, n, k):
    w, bits = Weight(n, k, fmt, 21), x_bits(tokens, k, 22)
    ref, tol = linear_ref(bits, w)
    assert_close(run_linear(bits, w), ref, tol, "fp32")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out_fp32", [True, False])
@pytest.mark.parametrize("beta,bias,gelu_on", [(0.0, True, True), (1.0, False, False),
                                               (-0.5, True, True), (0.0, False, True)])
def test_linear_epilogue_and_strides(fmt, out_fp32, beta, bias, gelu_on):
    t, n, k = 5, 224, 544
    w, bits = Weight(n, k, fmt, 31), x_bits(t, k, 32)
    rng = np.random.default_rng(33)
    b = rng.standard_normal(n).astype(np.float32) if bias else None
    y_in = rng.standard_normal((t, n)).astype(np.float32)
    y_in = bf16_bits_to_f64(synth.f32_to_bf16_bits(y_in)).astype(np.float32)
    acc, e = linear_ref(bits, w)
    pre = acc + beta * y_in + (b if bias else 0.0)
    ref = gelu(pre) if gelu_on else pre
    steps = 2.0 ** -22 * (np.abs(acc) + np.abs(beta * y_in) + (np.abs(b) if bias else 0) + np.abs(ref))
    tol = 1.13 * (e + steps) + 44 * 2.0 ** -24 * np.abs(ref)
    got = run_linear(bits, w, out_fp32, ld_x=k + 24, ld_y=n + 13, bias=b, beta=beta, gelu_on=gelu_on,
                     y_in=y_in if beta else None)
    assert_close(got, ref, tol + (0 if out_fp32 else ulp(ref)), "epilogue")


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_wide_ranges(fmt):
    """Activations whose groups differ by many binades, weights over the scales' whole range."""
    t, n, k = 6, 96, 1024
    lo, hi = (64, 190) if fmt == MX else (0, 0x7E)
    w = Weight(n, k, fmt, 41, lo, hi)
    x = bf16_bits_to_f64(x_bits(t, k, 42))
    x *= 2.0 ** np.repeat(np.arange(-28, 28, 7), 128)[None, :]
    x[1] *= 2.0 ** -60
    x[2, ::3] = 0.0
    x[3] = 0.0
    x[4, 128:] *= 2.0 ** np.random.default_rng(1).integers(-20, 1, k - 128)
    bits = synth.f32_to_bf16_bits(x.astype(np.float32))
    ref, tol = linear_ref(bits, w)
    got = run_linear(bits, w)
    assert_close(got, ref, tol, "ranges")
    assert (got[3] == 0).all()


def test_linear_scale_ends():
    """UE8M0 bytes 0 and 254, and 255 (NaN) in one block of one row."""
    n, k = 64, 256
    w = Weight(n, k, MX, 51, 127, 127)
    plain = np.full((n, k // 32), 127, dtype=np.uint8)
    plain[3, 2], plain[5, 7], plain[9, 0] = 0, 254, 255
    codes, _, _ = w.device()
    bits = x_bits(2, k, 52)
    bits[1] = synth.f32_to_bf16_bits(np.full((1, k), 2.0 ** 100, np.float32))[0]
    got = run_linear(bits, w, dev=(codes, dev_u8(oracle.scale_tile(plain)), None))
    v = oracle.e2m1_decode_array(w.codes, k).reshape(n, -1, 32)
    v = (v * np.exp2(plain.astype(np.float64) - 127)[:, :, None]).reshape(n, k)
    x = bf16_bits_to_f64(bits)
    ref, s = x @ v.T, np.abs(x) @ np.abs(v).T
    rows = [r for r in range(n) if r not in (9,)]
    big = np.abs(ref) > 3.4e38
    fine = ~big[:, rows]
    assert (np.abs(got[:, rows] - ref[:, rows])[fine] <= 1e-5 * s[:, rows][fine]).all()
    assert not np.isfinite(got[:, rows][~fine]).any()  # infinite weights of both signs
    assert np.isnan(got[:, 9]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_nonfinite_activations_stay_in_their_token(fmt):
    t, n, k = 9, 96, 416
    w, bits = Weight(n, k, fmt, 61), x_bits(t, k, 62)
    clean = run_linear(bits, w)
    bad = bits.copy()
    bad[2, 5], bad[4, 400], bad[8, 0] = 0x7FC0, 0x7F80, 0xFF80
    got = run_linear(bad, w)
    for r in range(t):
        if r == 2:
            assert np.isnan(got[r]).all()
        elif r in (4, 8):
            col = 400 if r == 4 else 0
            nz = w.value[:, col] != 0
            assert not np.isfinite(got[r]).any()
            sign = np.sign(w.value[nz, col]) * (1 if r == 4 else -1)
            assert (got[r][nz] == sign * np.inf).all() and np.isnan(got[r][~nz]).all()
        else:
            assert (got[r] == clean[r]).all()


def test_linear_offsets_past_32_bits():
    """Codes of 2^32 bytes and more: the last rows of a very tall weight."""
    n, k, t = (1 << 20) + 32, 8192 + 32, 1
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((mx.mx_scale_bytes(n, k, MX, TILED),), 120, dtype=torch.uint8, device="cuda")
    bits = x_bits(t, k, 72)
    y = guarded(n, torch.float32, float("nan"))
    mx.mx_linear_bf16(dev_bf16(bits), t, k, k, MX, codes, scales, None, n, y, n, mx.MX_OUT_FP32)
    torch.cuda.synchronize()
    check_guards(y)
    rows = np.r_[0:4, (1 << 19) - 2:(1 << 19) + 2, n - 40:n]
    v = oracle.e2m1_decode_array(codes[torch.from_numpy(rows).cuda()].cpu().numpy(), k) * 2.0 ** -7
    x = bf16_bits_to_f64(bits)
    tol = 1e-5 * (np.abs(x) @ np.abs(v).T) + fp16_loss(x, v)
    assert_close(y[torch.from_numpy(rows).cuda()].cpu().numpy()[None].astype(np.float64), x @ v.T, tol, "tall")
    assert torch.isfinite(y).all()


def test_linear_no_tokens_and_refusals():
    w = Weight(64, 64, MX, 81)
    codes, scales, _ = w.device()
    y = guarded(64, torch.float32, 7.0)
    x = dev_bf16(x_bits(1, 64, 82))
    mx.mx_linear_bf16(x, 0, 64, 64, MX, codes, scales, None, 64, y, 64, mx.MX_OUT_FP32)
    for kw, code in ((dict(tokens=33), mx.MX_ERR_UNSUPPORTED_SHAPE), (dict(k=48), mx.MX_ERR_UNSUPPORTED_SHAPE),
                     (dict(ld_x=32), mx.MX_ERR_INVALID_ARG), (dict(n=48), mx.MX_ERR_UNSUPPORTED_SHAPE)):
        a = dict(tokens=1, k=64, ld_x=64, n=64)
        a.update(kw)
        with pytest.raises(mx.MXError) as e:
            mx.mx_linear_bf16(x, a["tokens"], a["k"], a["ld_x"], MX, codes, scales, None, a["n"], y, 64,
                              mx.MX_OUT_FP32)
        assert e.value.code == code
    torch.cuda.synchronize()
    assert (y == 7.0).all()


# ---------------------------------------------------------------- the router

def run_route(bits, router_bits, bias, top_k, normalize, ld=None):
    t, h = bits.shape
    e = router_bits.shape[0]
    ids = guarded(t * top_k, torch.int32, 77)
    weights = guarded(t * top_k, torch.float32, float("nan"))
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    mx.mx_moe_route_bf16(strided(bits, ld or h), t, h, ld or h, dev_bf16(router_bits), e, b, top_k,
                         normalize, ids, weights)
    torch.cuda.synchronize()
    check_guards(ids, weights, what="route")
    return ids.view(t, top_k).cpu().numpy(), weights.view(t, top_k).cpu().numpy().astype(np.float64)


def route_ref(x, r, bias, top_k, normalize):
    l = x @ r.T + (0.0 if bias is None else bias.astype(np.float64))
    order = np.stack([np.lexsort((np.arange(l.shape[1]), -row)) for row in l])[:, :top_k]
    v = np.take_along_axis(l, order, 1)
    with np.errstate(invalid="ignore"):
        ex = np.exp(v - v[:, :1])
        norm = ex.sum(1) if normalize else np.exp(l - v[:, :1]).sum(1)
        w = ex / norm[:, None]
    none = np.isneginf(v)
    return np.where(none, -1, order), np.where(none, 0.0, w), l


@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("tokens,hidden,experts,top_k", [(1, 2048, 64, 8), (3, 32, 1, 1), (9, 96, 5, 5),
                                                         (64, 1056, 256, 8), (17, 4096, 512, 16),
                                                         (8, 544, 33, 2)])
def test_route(tokens, hidden, experts, top_k, normalize):
    bits = x_bits(tokens, hidden, 101)
    rb = synth.bf16_normal(experts, hidden, 1.5 * hidden ** -0.5, 102)
    ids, w = run_route(bits, rb, None, top_k, normalize, ld=hidden + 8)
    x, r = bf16_bits_to_f64(bits), bf16_bits_to_f64(rb)
    rid, rw, l = route_ref(x, r, None, top_k, normalize)
    err = 1e-6 * (np.abs(x) @ np.abs(r).T).max(1)
    s = -np.sort(-l, 1)
    for t in range(tokens):
        gaps = (s[t, :-1] - s[t, 1:])[:top_k]
        if gaps.size == 0 or gaps.min() > 2 * err[t]:
            assert (ids[t] == rid[t]).all()
            assert (np.abs(w[t] - rw[t]) <= (2e-5 + 2 * err[t]) * rw[t]).all()


def test_route_ties_take_the_lowest_index():
    """Small integers: every logit exact, many equal."""
    rng = np.random.default_rng(5)
    t, h, e, k = 40, 64, 200, 12
    x = rng.integers(-1, 2, (t, h)).astype(np.float32)
    r = rng.integers(-1, 2, (e, h)).astype(np.float32)
    r[100:] = r[:100]
    ids, w = run_route(synth.f32_to_bf16_bits(x), synth.f32_to_bf16_bits(r), None, k, 1)
    rid, rw, _ = route_ref(x.astype(np.float64), r.astype(np.float64), None, k, 1)
    assert (ids == rid).all()
    assert (np.abs(w - rw) <= 2e-5 * rw).all()


def test_route_masks():
    """-inf switches an expert off, the type's lowest value does not; too few experts leave empty
    slots; a NaN token has NaN weights and leaves the others alone."""
    rng = np.random.default_rng(6)
    t, h, e, k = 6, 96, 20, 4
    x, r = rng.integers(-2, 3, (t, h)).astype(np.float32), rng.integers(-2, 3, (e, h)).astype(np.float32)
    xb, rb = synth.f32_to_bf16_bits(x), synth.f32_to_bf16_bits(r)
    for bias in (np.where(np.arange(e) % 3 == 0, -np.inf, 0.0), np.where(np.arange(e) < 18, -np.inf, 0.0),
                 np.full(e, -np.inf), np.where(np.arange(e) < 18, np.finfo(np.float32).min, 0.0)):
        for normalize in (0, 1):
            ids, w = run_route(xb, rb, bias, k, normalize)
            l32 = (x.astype(np.float64) @ r.T.astype(np.float64)).astype(np.float32) + bias.astype(np.float32)
            rid, rw, _ = route_ref(np.eye(1), np.zeros((1, 1)), None, 1, 1)
            order = np.stack([np.lexsort((np.arange(e), -row)) for row in l32])[:, :k]
            v = np.take_along_axis(l32.astype(np.float64), order, 1)
            none = np.isneginf(v)
            assert (ids == np.where(none, -1, order)).all()
            with np.errstate(invalid="ignore"):
                ex = np.exp(v - v[:, :1])
                norm = (np.where(none, 0, ex) if normalize else np.exp(l32.astype(np.float64) - v[:, :1])).sum(1)
                rw = np.where(none, 0.0, ex / norm[:, None])
            assert (np.abs(w - rw) <= 2e-5 * rw).all()
    clean = run_route(xb, rb, None, k, 1)
    bad = xb.copy()
    bad[3, 7] = 0x7FC0
    ids, w = run_route(bad, rb, None, k, 1)
    assert np.isnan(w[3]).all() and (ids[3] == np.arange(k)).all()
    keep = [0, 1, 2, 4, 5]
    assert (ids[keep] == clean[0][keep]).all() and (w[keep] == clean[1][keep]).all()


# ---------------------------------------------------------------- the experts

class Layer:
    def __init__(self, experts, hidden, inter, fmt, act, seed):
        self.e, self.h, self.i, self.fmt, self.act = experts, hidden, inter, fmt, act
        self.gate, self.up = Stack(experts, inter, hidden, fmt, seed), Stack(experts, inter, hidden, fmt, seed + 1000)
        self.down = Stack(experts, hidden, inter, fmt, seed + 2000)
        self.moe = mx.moe_weights(fmt, experts, hidden, inter, self.gate.device, self.up.device,
                                  self.down.device, act)

    def ref(self, x, ids, weights):
        t = x.shape[0]
        y, tol, s = np.zeros((t, self.h)), np.zeros((t, self.h)), np.zeros((t, self.h))
        f = silu if self.act == mx.MX_ACT_SILU else gelu
        for r in range(t):
            for e, w in zip(ids[r], weights[r]):
                if e < 0 or e >= self.e:
                    continue
                wg, wu, wd = self.gate.w[e].value, self.up.w[e].value, self.down.w[e].value
                xr = x[r:r + 1]
                g, u = (xr @ wg.T)[0], (xr @ wu.T)[0]
                eg = 1e-5 * (np.abs(xr) @ np.abs(wg).T)[0] + fp16_loss(xr, wg)[0]
                eu = 1e-5 * (np.abs(xr) @ np.abs(wu).T)[0] + fp16_loss(xr, wu)[0]
                h = f(g) * u
                dh = 1.13 * eg * np.abs(u) + np.abs(f(g)) * eu + eg * eu + 2.0 ** -20 * np.abs(h)
                z = wd @ h
                dz = np.abs(wd) @ (dh + (2.0 ** -12 + 1e-5) * np.abs(h)) + fp16_loss(h[None], wd)[0]
                y[r] += w * z
                tol[r] += abs(w) * dz
                s[r] += abs(w) * np.abs(z)
        return y, tol + 2.0 ** -20 * s + ulp(y)


def run_experts(layer, bits, ids, weights, ld_x=None, ld_y=None, fill=0xFF):
    t, h = bits.shape
    top_k = ids.shape[1]
    ld_x, ld_y = ld_x or h, ld_y or h
    ws = guarded(mx.mx_moe_workspace_bytes(t, h, layer.i, top_k), torch.uint8, fill)
    body = guarded(t * ld_y, torch.bfloat16, float("nan"))
    y = body.view(t, ld_y)
    mx.mx_moe_experts_bf16(strided(bits, ld_x), t, ld_x, torch.from_numpy(ids.astype(np.int32)).cuda(),
                           torch.from_numpy(weights.astype(np.float32)).cuda(), top_k, layer.moe, y, ld_y, ws)
    torch.cuda.synchronize()
    check_guards(body, ws, what="experts")
    if ld_y > h:
        assert torch.isnan(y[:, h:].float()).all()
    return y[:, :h].float().cpu().numpy().astype(np.float64)


def choice(tokens, experts, top_k, seed, repeat=False):
    rng = np.random.default_rng(seed)
    ids = (rng.integers(0, experts, (tokens, top_k)) if repeat else
           np.stack([rng.permutation(experts)[:top_k] for _ in range(tokens)]))
    w = rng.random((tokens, top_k)).astype(np.float32) + np.float32(0.05)
    return ids.astype(np.int32), w


SIZES = [(1, 256, 128, 4, 2), (3, 544, 96, 7, 3), (8, 160, 288, 9, 4), (17, 1056, 416, 6, 6),
         (64, 128, 160, 16, 8), (2, 2080, 1568, 3, 1), (5, 32, 32, 5, 2), (33, 256, 256, 2, 1)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", [mx.MX_ACT_SILU, mx.MX_ACT_GELU])
@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k", SIZES)
def test_experts(fmt, act, tokens, hidden, inter, experts, top_k):
    layer = Layer(experts, hidden, inter, fmt, act, 201)
    bits = x_bits(tokens, hidden, 202)
    ids, w = choice(tokens, experts, top_k, 203)
    ref, tol = layer.ref(bf16_bits_to_f64(bits), ids, w)
    got = run_experts(layer, bits, ids, w, ld_x=hidden + 16, ld_y=hidden + 5)
    assert_close(got, ref, tol, "experts")


@pytest.mark.parametrize("fmt", FMTS)
def test_experts_empty_repeated_and_crowded_slots(fmt):
    layer = Layer(6, 288, 160, fmt, mx.MX_ACT_SILU, 301)
    for tokens in (1, 4, 11, 64):
        bits = x_bits(tokens, 288, 302)
        x = bf16_bits_to_f64(bits)
        ids, w = choice(tokens, 6, 4, 303, repeat=True)
        cases = {"repeated": ids}
        some = ids.copy()
        some[np.random.default_rng(4).random(some.shape) < 0.4] = -1
        some[-1] = [-1, 6, 1 << 30, -(1 << 31)]
        cases["empty"] = some
        cases["none"] = np.full_like(ids, -1)
        cases["one expert"] = np.full_like(ids, 5)
        for name, c in cases.items():
            ref, tol = layer.ref(x, c, w)
            got = run_experts(layer, bits, c, w)
            assert_close(got, ref, tol, f"{name} {tokens}")
            empty = ((c < 0) | (c >= 6)).all(1)
            assert (got[empty] == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_experts_many(fmt):
    """512 experts, 16 slots, offsets past 2^31 bytes of codes in a stack."""
    e, h, i = 512, 4096 + 32, 2048 + 32
    blk = block(fmt)
    g = torch.Generator(device="cuda").manual_seed(9)
    stacks = []
    for rows, k in ((i, h), (i, h), (h, i)):
        codes = torch.randint(0, 256, (e, rows, k // 2), generator=g, dtype=torch.uint8, device="cuda")
        sb = mx.mx_scale_bytes(rows, k, fmt, TILED)
        scales = torch.full((e, sb), 119 if fmt == MX else 0x38, dtype=torch.uint8, device="cuda")
        ts = None if fmt == MX else torch.full((e,), 2.0 ** -8, dtype=torch.float32, device="cuda")
        stacks.append((codes, scales, ts))
    moe = mx.moe_weights(fmt, e, h, i, *stacks)
    t, top_k = 2, 16
    bits = x_bits(t, h, 402)
    ids = np.stack([np.r_[511, 0, 510, np.arange(300, 313)], np.r_[509, 511, np.arange(480, 494)]]).astype(np.int32)
    w = np.full((t, top_k), 0.25, np.float32)
    ws = guarded(mx.mx_moe_workspace_bytes(t, h, i, top_k), torch.uint8, 0xFF)
    y = guarded(t * h, torch.bfloat16, float("nan")).view(t, h)
    mx.mx_moe_experts_bf16(dev_bf16(bits), t, h, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(),
                           top_k, moe, y, h, ws)
    x = torch.from_numpy(bf16_bits_to_f64(bits)).cuda()
    table = torch.tensor([oracle.e2m1_decode(c) for c in range(16)], dtype=torch.float64, device="cuda")
    unit = 2.0 ** -8  # 2^(119 - 127), or E4M3 0x38 = 1 times 2^-8

    def value(s, idx):
        c = stacks[s][0][idx].long()
        return torch.stack([table[c & 15], table[c >> 4]], -1).reshape(c.shape[0], -1) * unit

    assert blk * (h // blk) == h
    ref, mag = torch.zeros((t, h), dtype=torch.float64, device="cuda"), torch.zeros((t, h), dtype=torch.float64, device="cuda")
    for r in range(t):
        for idx, wt in zip(ids[r], w[r]):
            a, b = value(0, idx) @ x[r], value(1, idx) @ x[r]
            hv = a * torch.sigmoid(a) * b
            d = value(2, idx)
            ref[r] += float(wt) * (d @ hv)
            # h to 2^-12 in the second product and 1e-5 of the sums, twice over
            sg, su = value(0, idx).abs() @ x[r].abs(), value(1, idx).abs() @ x[r].abs()
            dh = 2.0 ** -12 * hv.abs() + 2e-5 * (1.13 * sg * b.abs() + (a * torch.sigmoid(a)).abs() * su)
            mag[r] += float(wt) * (d.abs() @ (dh + 2e-5 * hv.abs()))
    ref, mag = ref.cpu().numpy(), mag.cpu().numpy()
    assert_close(y.float().cpu().numpy().astype(np.float64), ref, mag + 1.01 * ulp(ref), "many experts")


def test_experts_nonfinite_token_and_tensor_scales():
    layer = Layer(4, 96, 64, NV, mx.MX_ACT_SILU, 501)
    bits = x_bits(5, 96, 502)
    ids, w = choice(5, 4, 2, 503)
    clean = run_experts(layer, bits, ids, w)
    bad = bits.copy()
    bad[1, 3] = 0x7FC0
    got = run_experts(layer, bad, ids, w)
    assert np.isnan(got[1]).all()
    keep = [0, 2, 3, 4]
    assert (got[keep] == clean[keep]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [1, 6, 24, 64])
def test_layer_equals_its_parts(fmt, tokens):
    """mx_moe_layer_bf16 is mx_moe_route_bf16 and then mx_moe_experts_bf16, bit for bit, twice over."""
    h, i, e, k = 416, 224, 12, 3
    layer = Layer(e, h, i, fmt, mx.MX_ACT_SILU, 601)
    bits = x_bits(tokens, h, 602)
    rb = synth.bf16_normal(e, h, 1.5 * h ** -0.5, 603)
    bias = np.where(np.arange(e) == 4, -np.inf, 0.0)
    ids, w = run_route(bits, rb, bias, k, 1)
    want = run_experts(layer, bits, ids, w)
    x, r, b = dev_bf16(bits), dev_bf16(rb), torch.from_numpy(bias.astype(np.float32)).cuda()
    for fill in (0x00, 0xFF):
        ws = guarded(mx.mx_moe_workspace_bytes(tokens, h, i, k), torch.uint8, fill)
        gi, gw = guarded(tokens * k, torch.int32, 5), guarded(tokens * k, torch.float32, 0.5)
        y = guarded(tokens * h, torch.bfloat16, float("nan"))
        mx.mx_moe_layer_bf16(x, tokens, h, r, b, k, True, layer.moe, gi, gw, y, h, ws)
        torch.cuda.synchronize()
        check_guards(ws, gi, gw, y, what="layer")
        assert (gi.view(tokens, k).cpu().numpy() == ids).all()
        assert (gw.view(tokens, k).cpu().numpy().astype(np.float64) == w).all()
        assert (y.view(tokens, h).float().cpu().numpy().astype(np.float64) == want).all()


def test_streams_graph_and_repeats():
    """On another stream, in a graph replayed on new inputs, and again: the same bits."""
    h, i, e, k, t = 544, 320, 8, 3, 7
    layer = Layer(e, h, i, MX, mx.MX_ACT_GELU, 701)
    w = Weight(288, h, NV, 702)
    codes, scales, ts = w.device()
    rb = dev_bf16(synth.bf16_normal(e, h, 1.5 * h ** -0.5, 703))
    xs = [dev_bf16(x_bits(t, h, 704 + j)) for j in range(3)]
    x = torch.empty_like(xs[0])
    ws = torch.empty(mx.mx_moe_workspace_bytes(t, h, i, k), dtype=torch.uint8, device="cuda")
    ids = torch.empty((t, k), dtype=torch.int32, device="cuda")
    wt = torch.empty((t, k), dtype=torch.float32, device="cuda")
    y = torch.empty((t, h), dtype=torch.bfloat16, device="cuda")
    z = torch.empty((t, 288), dtype=torch.float32, device="cuda")

    def step():
        mx.mx_moe_layer_bf16(x, t, h, rb, None, k, False, layer.moe, ids, wt, y, h, ws)
        mx.mx_linear_bf16(y, t, h, h, NV, codes, scales, ts, 288, z, 288, mx.MX_OUT_FP32)

    want = []
    for v in xs:
        x.copy_(v)
        step()
        torch.cuda.synchronize()
        want.append((ids.clone(), wt.clone(), y.clone(), z.clone()))
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        with torch.cuda.graph(g, stream=s):
            step()
        for j in (1, 0, 2, 2):
            x.copy_(xs[j])
            for b in (y, z):
                b.fill_(float("nan"))
            g.replay()
            got = (ids.clone(), wt.clone(), y.clone(), z.clone())
            s.synchronize()
            for a, b in zip(got, want[j]):
                assert torch.equal(a, b)
    assert mx.mx_device_status() == mx.MX_OK
