"""The decoding step's operators in binary64, from their formulas (numpy)."""
from __future__ import annotations

import numpy as np

BLOCK = 32


def bf16_round(x):
    """binary32/64 values rounded to BF16 (nearest even), as binary64."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return r.astype(np.uint32).view(np.float32).astype(np.float64)


# ---------------------------------------------------------------- norm and rotation

def pairs(rotary, interleaved):
    i = np.arange(rotary // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)


def rotate(x, positions, inv_freq, rotary, interleaved, sign=1.0):
    """x [tokens, heads, dim] turned by its positions."""
    y = x.copy()
    if rotary:
        phi = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]
        c, s = np.cos(phi)[:, None], sign * np.sin(phi)[:, None]
        i, j = pairs(rotary, interleaved)
        y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    return y


def norm_rotate(x, w, eps, positions, inv_freq, rotary, interleaved):
    n = x if w is None else x * w / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(n, positions, inv_freq, rotary, interleaved)


def norm_rotate_backward(x, dy, w, eps, positions, inv_freq, rotary, interleaved):
    """(dx, dw, size of dx's terms, size of dw's terms)."""
    g = rotate(dy, positions, inv_freq, rotary, interleaved, -1.0)
    size = rotate_size(dy, rotary, interleaved)
    if w is None:
        return g, None, size, None
    d = x.shape[-1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n, gw = x * r, g * w
    dx = r * (gw - n * (gw * n).sum(-1, keepdims=True) / d)
    dx_size = r * (size * abs(w) + abs(n) * (size * abs(w) * abs(n)).sum(-1, keepdims=True) / d)
    return dx, (g * n).sum((0, 1)), dx_size, (size * abs(n)).sum((0, 1))


def rotate_size(x, rotary, interleaved):
    """|a| + |b| for the channels of a pair (a, b), |x| for the others."""
    y = abs(x)
    if rotary:
        i, j = pairs(rotary, interleaved)
        y[..., i] = y[..., j] = abs(x[..., i]) + abs(x[..., j])
    return y


# ---------------------------------------------------------------- cache

def e4m3_table():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


E4M3 = e4m3_table()


def e4m3_round(v):
    """binary64 to E4M3 bytes: nearest even, at most 448, infinities and NaN to NaN (0x7F)."""
    a = np.where(np.isfinite(v), np.abs(v), 0.0)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    a = np.minimum(np.rint(a / np.exp2(e - 3)) * np.exp2(e - 3), 448.0)
    code = np.searchsorted(E4M3[:127], a).astype(np.uint8)
    code = np.where(np.signbit(v), code | 0x80, code).astype(np.uint8)
    return np.where(np.isfinite(v), code, 0x7F).astype(np.uint8)


def block_exponent(amax):
    """The least e in -127 .. 127 with amax <= 448 * 2^e (-127 for 0)."""
    for e in range(-127, 128):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return 127


class Cache:
    """A pool of pages, its page table and lengths; codes and scales as the C structure has them."""

    def __init__(self, pages, page_tokens, heads, dim, table, seed=0):
        rng = np.random.default_rng(seed)
        self.pages, self.page_tokens, self.heads, self.dim = pages, page_tokens, heads, dim
        self.table = np.asarray(table, np.int32)
        self.codes = [rng.integers(0, 256, (pages, heads, page_tokens, dim)).astype(np.uint8) for _ in range(2)]
        self.scales = [rng.integers(0, 255, (pages, heads, page_tokens // BLOCK)).astype(np.uint8)
                       for _ in range(2)]

    def append(self, new, counts, lengths):
        """new: (k, v) [tokens, heads, dim]; the rows of sequence b follow those of b - 1."""
        for which in range(2):
            row = 0
            for b, n in enumerate(counts):
                for i in range(n):
                    self._put(which, b, int(lengths[b]) - n, i, n, new[which], row)
                row += n

    def _put(self, which, b, first, i, n, x, row):
        """Block by block: does the work for the first stored token i of each block."""
        pos = first + i
        if pos < 0 or (i > 0 and first + i - 1 >= 0 and pos % BLOCK != 0):
            return
        page_index = pos // self.page_tokens
        page = self.table[b, page_index] if page_index < self.table.shape[1] else -1
        if not 0 <= page < self.pages:
            return
        off = pos % self.page_tokens
        block, held = off // BLOCK, off % BLOCK
        m = min(BLOCK - held, n - i)
        for h in range(self.heads):
            v = x[row + i:row + i + m, h]
            fin = np.abs(v[np.isfinite(v)])
            e = block_exponent(fin.max() if fin.size else 0.0)
            codes = self.codes[which][page, h, block * BLOCK:(block + 1) * BLOCK]
            if held:
                old = int(self.scales[which][page, h, block]) - 127
                if e > old:
                    codes[:held] = e4m3_round_codes(codes[:held], old - e)
                e = max(e, old)
            codes[held:held + m] = e4m3_round(v * 2.0 ** -e)
            self.scales[which][page, h, block] = e + 127

    def values(self, which, b, length):
        """binary64 [length, heads, dim] of sequence b; rows of bad pages are None-marked by `ok`."""
        out = np.zeros((length, self.heads, self.dim))
        ok = np.zeros(length, bool)
        for t in range(length):
            page = self.table[b, t // self.page_tokens]
            if not 0 <= page < self.pages:
                continue
            off = t % self.page_tokens
            s = 2.0 ** (self.scales[which][page, :, off // BLOCK].astype(np.float64) - 127)
            out[t] = E4M3[self.codes[which][page, :, off]] * s[:, None]
            ok[t] = True
        return out, ok


def e4m3_round_codes(codes, shift):
    """Codes under a scale 2^-shift times as large."""
    v = E4M3[codes] * 2.0 ** shift
    out = e4m3_round(v)
    return np.where((codes & 0x7F) == 0x7F, codes, out)


def attention(cache, q, lengths, q_tokens, q_heads, scale, window):
    """out, lse and an error bound of each, all [rows, q_heads, ...], for q [rows, q_heads, dim].

    Bound of out before its own rounding: a logit is off by at most dl = (dim + 8) 2^-24 scale
    sum |q||k| (binary32 sums) + 2^-21 (|logit| + 1) (its scaling and the exponential), a weight
    by 2 dl (its own and its sum's) + 2^-11 (FP16) + 2^-18 + tokens 2^-27 (sums over 16 tokens at a
    time, 2^-23 each).  FP16 weights are lifted so that the row's largest weight * value scale
    comes to at least 2^13: those below 2^-14 are off by up to 2^-25, 2^-38 of that largest, times the
    value's code; of lse dl + 2^-18."""
    group = q_heads // cache.heads
    rows = q.shape[0]
    out, lse = np.zeros((rows, q_heads, cache.dim)), np.full((rows, q_heads), -np.inf)
    e_out, e_lse = np.zeros_like(out), np.zeros_like(lse)
    for b, length in enumerate(lengths):
        length = int(length)
        if length <= 0:
            continue
        k, ok = cache.values(0, b, length)
        v, _ = cache.values(1, b, length)
        t = np.arange(length)
        unit = np.zeros((length, cache.heads))  # scale of each value
        for x in range(length):
            page, off = cache.table[b, x // cache.page_tokens], x % cache.page_tokens
            if ok[x]:
                unit[x] = 2.0 ** (cache.scales[1][page, :, off // BLOCK].astype(np.float64) - 127)
        for i in range(q_tokens):
            p = length - q_tokens + i
            see = ok & (t <= p)
            if window:
                see &= t > p - window
            if not see.any():
                continue
            for h in range(q_heads):
                kk, vv = k[see, h // group], v[see, h // group]
                x = q[b * q_tokens + i, h]
                l = scale * (kk @ x)
                top = l.max()
                w = np.exp(l - top)
                total = w.sum()
                r = b * q_tokens + i
                out[r, h] = w @ vv / total
                lse[r, h] = top + np.log(total)
                dl = ((cache.dim + 8) * 2.0 ** -24 * abs(scale) * (np.abs(kk) @ np.abs(x)) +
                      2.0 ** -21 * (np.abs(l) + 1)).max()
                u = unit[see, h // group]
                small = 2.0 ** -38 * (w * u).max() * (np.abs(vv) / u[:, None]).sum(0)
                rel = 2 * dl + 2.0 ** -11 + 2.0 ** -18 + len(w) * 2.0 ** -27
                e_out[r, h] = (rel * (w @ np.abs(vv)) + small) / total
                e_lse[r, h] = dl + 2.0 ** -18
    return out, lse, e_out, e_lse


# ---------------------------------------------------------------- sampling

def sample(logits, temperature, top_k, top_p, min_p, uniform):
    """(id, probability, how near the nearest border that decided it is)."""
    l = np.asarray(logits, np.float64)
    if np.isnan(l).any() or any(np.isnan(v) for v in (temperature, top_p, min_p, uniform)) or l.max() == -np.inf:
        return -1, 0.0, 1.0
    order = np.argsort(-l, kind="stable")
    if temperature <= 0:
        return int(order[0]), 1.0, 1.0
    d = np.where(l[order] == l[order[0]], 0.0, l[order] - l[order[0]])
    with np.errstate(over="ignore"):
        w = np.exp(d / max(float(temperature), 2.0 ** -100))
    if 0 < top_k < len(w):
        w[top_k:] = 0
    near = 1.0
    if top_p < 1:
        cum = np.cumsum(w)
        n = max(1, int(np.searchsorted(cum, top_p * cum[-1], side="left")) + 1) if top_p > 0 else 1
        if top_p > 0:
            near = min(near, np.abs(cum / cum[-1] - top_p).min())
        w[n:] = 0
    if min_p > 0:
        rel = np.abs(w / min(float(min_p), 1.0) - 1)
        near = min(near, rel[1:].min() if len(rel) > 1 else 1.0)
        w[1:][w[1:] < min_p] = 0
    kept = np.zeros_like(w)
    kept[order] = w
    cum = np.cumsum(kept)
    u = min(max(float(uniform), 0.0), float(np.float32(1) - np.float32(2) ** -24))
    i = int(np.searchsorted(cum, u * cum[-1], side="right"))
    i = min(i, int(np.nonzero(kept)[0][-1]))
    near = min(near, np.abs(cum / cum[-1] - u)[kept > 0].min()) if u > 0 else near
    return i, kept[i] / cum[-1], near
