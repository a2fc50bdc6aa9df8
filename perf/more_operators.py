"""The rest of a decoding step beside its FP4 products, measured.

Five operators, one pass each:

* rotate:  RMS norm of every query and key head and the rotation by position;
* back:    its gradients (inputs and norm weights);
* append:  new keys and values into a paged cache of E4M3 codes with a UE8M0 scale for each
           32 tokens of a page and head;
* attend:  a few query tokens of each sequence over that cache;
* sample:  the next token by temperature, top-k, top-p and min-p from a given random number.

`own` chooses between the plain forms below (elementary torch operations in binary32, in
binary64 for angles, long sums and the choice of a token) and the calls of the package.
"""
import numpy as np
import torch

own = False

BLOCK = 32  # tokens of a scale
PAGE = 64   # tokens of a page
PER_PAGE = PAGE // BLOCK


# ---------------------------------------------------------------- cases

def _named(name, c):
    return dict(c, name=name) if name else c


def rotate(name, op, tokens, q_heads, k_heads, head_dim, rotary_dim, interleaved, far):
    return _named(name, dict(op=op, tokens=tokens, q_heads=q_heads, k_heads=k_heads, head_dim=head_dim,
                             rotary_dim=rotary_dim, interleaved=interleaved, far=far))


def append(name, sequences, tokens, kv_heads, head_dim, held):
    """`tokens` new ones in all, behind up to `held` that a sequence has; one each where they are as many."""
    return _named(name, dict(op="append", sequences=sequences, tokens=tokens, kv_heads=kv_heads,
                             head_dim=head_dim, held=held))


def attend(name, sequences, q_tokens, length, q_heads, kv_heads, head_dim, window=0, lse=False):
    return _named(name, dict(op="attend", sequences=sequences, q_tokens=q_tokens, length=length,
                             q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, window=window, lse=lse))


def sample(name, rows, vocab, dtype, mode):
    return _named(name, dict(op="sample", rows=rows, vocab=vocab, dtype=dtype, mode=mode))


def listed():
    return [
        # one sequence decoding: launch and latency count
        rotate("rotate 1x(32+8)x128", "rotate", 1, 32, 8, 128, 128, False, 100000),
        # a long prompt, half of each head rotated
        rotate("rotate 8192x(64+8)x128 half", "rotate", 8192, 64, 8, 128, 64, False, 8192),
        # a small training batch, neighbouring channels paired, an odd number of tokens
        rotate("back 333x(12+4)x64 pairs", "back", 333, 12, 4, 64, 64, True, 4096),
        # a training step's layer
        rotate("back 4096x(32+8)x128", "back", 4096, 32, 8, 128, 128, False, 4096),
        # a decode batch: one token each behind what is held, some scales grow
        append("append 64x1 8x128", 64, 64, 8, 128, 1024),
        # prompts of several sequences together, none of a round length
        append("append 8 of 16384 8x128", 8, 16384, 8, 128, 100),
        # one sequence: latency
        attend("attend 1x1x4096 32/8x128", 1, 1, 4096, 32, 8, 128),
        # a decode batch of uneven lengths
        attend("attend 64x1x8192 64/8x128", 64, 1, 8192, 64, 8, 128),
        # one long context, few heads of keys
        attend("attend 1x1x131072 32/4x128", 1, 1, 131072, 32, 4, 128),
        # drafts of four tokens, a window, an odd group, small heads, log-sum-exp out
        attend("attend 7x4x5000 28/4x64 window", 7, 4, 5000, 28, 4, 64, window=1000, lse=True),
        # one row, a short list of candidates
        sample("sample 1x32000 top-k", 1, 32000, "fp32", "top_k"),
        # a decode batch whose rows want different things
        sample("sample 64x131072 mixed", 64, 131072, "fp32", "mixed"),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["rotate", "back", "append", "attend", "attend", "sample", "sample"])
    if op in ("rotate", "back"):
        dim = rng.choice([48, 64, 80, 96, 128, 128, 192, 256])
        q, k = _log_int(rng, 1, 64), _log_int(rng, 1, 16)
        most = (8192 * 72 * 128 if op == "rotate" else 4096 * 40 * 128) // ((q + k) * dim)
        return rotate(None, op, min(_log_int(rng, 1, 8192), most), q, k, dim, 16 * rng.randint(1, dim // 16),
                      rng.random() < 0.5, _log_int(rng, 100, 1000000))
    if op == "append":
        heads, dim = rng.choice([1, 2, 4, 8, 10]), rng.choice([64, 128, 256])
        sequences = _log_int(rng, 1, 128)
        most = 16384 * 8 * 128 // (heads * dim)
        tokens = sequences if rng.random() < 0.5 else min(most, sequences * _log_int(rng, 1, 4000) + rng.randint(1, 31))
        return append(None, sequences, max(tokens, sequences), heads, dim, _log_int(rng, 1, 2000))
    if op == "attend":
        heads, dim, sequences = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256]), _log_int(rng, 1, 100)
        length = _log_int(rng, 1, min(131072, 64 * 8192 * 8 * 128 // (sequences * heads * dim)))
        q_tokens = rng.choice([1, 1, 1, 2, 3, 5, 8])
        return attend(None, sequences, q_tokens, max(length, q_tokens), heads * rng.randint(1, 12), heads, dim,
                      rng.choice([0, 0, _log_int(rng, 10, 4096)]), rng.random() < 0.3)
    rows = _log_int(rng, 1, 256)
    vocab = _log_int(rng, 1000, min(262144, 64 * 131072 // rows))
    return sample(None, rows, vocab, rng.choice(["fp32", "bf16"]), rng.choice(["plain", "top_k", "top_p", "min_p", "mixed"]))


# ---------------------------------------------------------------- inputs

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(shape, g):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _heads(g, tokens, heads, dim):
    """A projection's heads: channels and heads of different spread."""
    return (_randn((tokens, heads, dim), g) * (0.3 + 1.5 * _rand((1, heads, dim), g))).to(torch.bfloat16)


def _prepare_rotate(c, g):
    t, q, k, d, r = c["tokens"], c["q_heads"], c["k_heads"], c["head_dim"], c["rotary_dim"]
    # queries and keys lie in one row, as a fused projection writes them
    s = {"x": torch.cat([_heads(g, t, q, d), _heads(g, t, k, d)], 1).reshape(t, (q + k) * d)}
    s["q_weight"] = (1.0 + 0.2 * _randn((d,), g)).to(torch.bfloat16)
    s["k_weight"] = (1.0 + 0.2 * _randn((d,), g)).to(torch.bfloat16)
    s["inv_freq"] = (10000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)).float()
    s["positions"] = (torch.arange(t, device="cuda") + (_rand((t,), g) * c["far"]).long()).to(torch.int32)
    s["eps"] = 1e-6
    s["y"] = torch.empty_like(s["x"])
    if c["op"] == "back":
        s["dy"] = (_randn((t, (q + k) * d), g) * 0.01).to(torch.bfloat16)
        s["dq_weight"] = torch.empty(d, device="cuda")
        s["dk_weight"] = torch.empty(d, device="cuda")
    return s


def _quantize(x, e):
    """E4M3 codes of x under scales 2^e."""
    return torch.ldexp(x, -e).to(torch.float8_e4m3fn)


def _exponent(amax):
    """The least e with amax <= 448 2^e (-127 for zero)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    return torch.where(amax == 0, torch.full_like(e, -127), e - 9 + (m > 0.875)).clamp(-127, 127)


def _pool(g, pages, heads, dim, spread):
    """A pool of pages: E4M3 codes [pages, heads, PAGE, dim], UE8M0 bytes [pages, heads, PAGE / BLOCK]."""
    x = _randn((pages, heads, PER_PAGE, BLOCK, dim), g)
    x *= torch.exp2(spread * _randn((pages, heads, PER_PAGE, 1, 1), g))
    e = _exponent(x.abs().amax((-1, -2)))
    codes = _quantize(x, e[..., None, None]).view(torch.uint8).view(pages, heads, PAGE, dim)
    return codes, (e + 127).to(torch.uint8)


def _pages(g, s, lengths, total):
    """A page table for sequences of these lengths, of scattered pages of a pool of `total`."""
    need = max(1, -(-int(lengths.max()) // PAGE))
    used = -(-lengths // PAGE)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(need, device="cuda")[None]
    first = (torch.cumsum(used, 0) - used)[:, None]
    # entries behind a sequence's end are never read
    s["page_table"] = torch.where(at < used[:, None], order[(first + at).clamp(max=total - 1)], -1).to(torch.int32)
    s["lengths"] = lengths.to(torch.int32)


def _prepare_append(c, g):
    b, t, h, d = c["sequences"], c["tokens"], c["kv_heads"], c["head_dim"]
    if t == b:
        counts = torch.ones(b, dtype=torch.int64, device="cuda")
    else:  # prompts of uneven lengths
        share = _rand((b,), g) + 0.1
        ends = (torch.cumsum(share, 0) / share.sum() * (t - b)).long()
        ends[-1] = t - b
        counts = torch.diff(ends, prepend=ends.new_zeros(1)) + 1
    held = (_rand((b,), g) * (c["held"] + 1)).long()
    s = {"starts": torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).to(torch.int32)}
    s["pages"] = (t + b * c["held"]) // PAGE + 2 * b + 3  # (a few belong to nobody)
    _pages(g, s, held + counts, s["pages"])
    s["k_codes"], s["k_scales"] = _pool(g, s["pages"], h, d, 0.5)
    s["v_codes"], s["v_scales"] = _pool(g, s["pages"], h, d, 0.5)
    grown = 1.0 + 7.0 * (_rand((t, 1, 1), g) < 0.1)  # some outgrow the scale that a block has
    s["k"] = (_randn((t, h, d), g) * grown).to(torch.bfloat16).view(t, h * d)
    s["v"] = (_randn((t, h, d), g) * grown).to(torch.bfloat16).view(t, h * d)
    return s


def _prepare_attend(c, g):
    b, n, h, d = c["sequences"], c["q_tokens"], c["kv_heads"], c["head_dim"]
    lengths = (c["length"] * (0.1 + 0.9 * _rand((b,), g))).long().clamp(min=n)
    lengths[0] = c["length"]
    if b > 4:
        lengths[-1] = 0  # a slot of the batch that is empty
    s = {"pages": int((-(-lengths // PAGE)).sum()) + 3}  # (a few belong to nobody)
    _pages(g, s, lengths, s["pages"])
    s["k_codes"], s["k_scales"] = _pool(g, s["pages"], h, d, 0.0)
    s["v_codes"], s["v_scales"] = _pool(g, s["pages"], h, d, 1.0)
    s["q"] = (2.0 * _randn((b * n, c["q_heads"] * d), g)).to(torch.bfloat16)
    s["scale"] = d ** -0.5
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((b * n, c["q_heads"]), device="cuda") if c["lse"] else None
    return s


def _prepare_sample(c, g):
    n, v, mode = c["rows"], c["vocab"], c["mode"]
    x = _randn((n, v), g) * (1.5 + 1.5 * _rand((n, 1), g))
    x += 5.0 * (_rand((n, v), g) < 20.0 / v)  # a few likely tokens
    x[:, v - v // 50:] = float("-inf")       # the padding of the vocabulary, switched off
    s = {"logits": x.to(torch.float32 if c["dtype"] == "fp32" else torch.bfloat16)}
    pick = torch.arange(n, device="cuda") % 5  # mixed: what each row wants
    on = lambda name, k: (pick == k) | (pick == 4) if mode == "mixed" else pick.new_full((n,), mode == name).bool()  # noqa: E731
    s["temperature"] = 0.5 + _rand((n,), g)
    if mode == "mixed":
        s["temperature"][pick == 3] = 0.0
    s["top_k"] = torch.where(on("top_k", 0), (2.0 ** (1.0 + 8.0 * _rand((n,), g))).int(), 0).to(torch.int32)
    s["top_p"] = torch.where(on("top_p", 1), 0.8 + 0.19 * _rand((n,), g), 1.0)
    s["min_p"] = torch.where(on("min_p", 2), 0.02 + 0.1 * _rand((n,), g), 0.0)
    s["uniform"] = _rand((n,), g)
    s["ids"] = torch.empty(n, dtype=torch.int32, device="cuda")
    s["probability"] = torch.empty(n, device="cuda")
    return s


def prepare(case, seed):
    make = {"rotate": _prepare_rotate, "back": _prepare_rotate, "append": _prepare_append,
            "attend": _prepare_attend, "sample": _prepare_sample}[case["op"]]
    return dict(make(case, _rng(seed)), case=dict(case))


# ---------------------------------------------------------------- plain forms

def _split(x, c):
    """[tokens, (q + k) dim] to [tokens, q + k, dim] in binary32."""
    return x.float().view(c["tokens"], -1, c["head_dim"])


def _weights(s, c):
    """The norm weights of every head, [q + k, dim]."""
    q, k = (s[n].float()[None].expand(c[m], -1) for n, m in (("q_weight", "q_heads"), ("k_weight", "k_heads")))
    return torch.cat([q, k])


def _turn(x, s, c, sign):
    """The rotation of x [tokens, heads, dim] by its positions (sign -1: back)."""
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None]
    cos, sin = torch.cos(angle).float()[:, None], sign * torch.sin(angle).float()[:, None]
    r = c["rotary_dim"]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_rotate(s):
    c = s["case"]
    x = _split(s["x"], c)
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * _weights(s, c)
    y = _turn(n, s, c, 1.0).to(torch.bfloat16)
    return {"q": y[:, :c["q_heads"]], "k": y[:, c["q_heads"]:]}


def _plain_back(s):
    c, q = s["case"], s["case"]["q_heads"]
    x, dy = _split(s["x"], c), _split(s["dy"], c)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    g, n = _turn(dy, s, c, -1.0), x * r
    dw = (g * n).sum(0, dtype=torch.float64)
    gw = g * _weights(s, c)
    dx = (r * (gw - n * (gw * n).mean(-1, keepdim=True))).to(torch.bfloat16)
    return {"dq": dx[:, :q], "dk": dx[:, q:], "dq_weight": dw[:q].sum(0).float(), "dk_weight": dw[q:].sum(0).float()}


def _plain_store(s, x, codes, scales):
    """New rows x into one of the pools, where their sequences go on."""
    c = s["case"]
    t, h, d = c["tokens"], c["kv_heads"], c["head_dim"]
    starts, lengths = s["starts"].long(), s["lengths"].long()
    counts = starts[1:] - starts[:-1]
    first = lengths - counts
    seq = torch.bucketize(torch.arange(t, device=x.device), starts[1:], right=True)
    pos = first[seq] + torch.arange(t, device=x.device) - starts[seq]
    at = s["page_table"].long()[seq, pos // PAGE] * PER_PAGE + pos % PAGE // BLOCK  # block of each new row
    x = x.float().view(t, h, d)
    amax = torch.zeros((scales.shape[0] * PER_PAGE, h), device=x.device)
    amax.scatter_reduce_(0, at[:, None].expand(-1, h), x.abs().amax(-1), "amax")
    e = _exponent(amax)
    # the block that a sequence goes on in keeps at least its scale, and what it holds is rounded again where that grows
    page0, block0 = s["page_table"].long().gather(1, first[:, None] // PAGE)[:, 0], first % PAGE // BLOCK
    at0, off = page0 * PER_PAGE + block0, first % BLOCK
    before = torch.where(off[:, None] > 0, scales[page0, :, block0].to(e.dtype) - 127, -127)
    e[at0] = torch.maximum(e[at0], before)
    blocks = codes.view(-1, h, PER_PAGE, BLOCK, d)
    held = blocks[page0, :, block0]  # [sequences, heads, token, dim]
    again = _quantize(held.view(torch.float8_e4m3fn).float(), (e[at0] - before)[..., None, None]).view(torch.uint8)
    old = (torch.arange(BLOCK, device=x.device)[None] < off[:, None])[:, None, :, None]
    blocks[page0, :, block0] = torch.where(old, again, held)
    new = _quantize(x, e[at][..., None]).view(torch.uint8)
    codes[at // PER_PAGE, :, pos % PAGE] = new
    touched = torch.zeros(e.shape[0], dtype=torch.bool, device=x.device)
    touched[at] = True
    byte = (e + 127).to(torch.uint8).view(-1, PER_PAGE, h).transpose(1, 2)
    scales.copy_(torch.where(touched.view(-1, 1, PER_PAGE), byte, scales))


def _cache_out(s):
    """The pools as the numbers that they hold: codes, and the scales beside them."""
    return {n: s[n].view(torch.float8_e4m3fn if n.endswith("codes") else torch.float8_e8m0fnu)
            for n in ("k_codes", "k_scales", "v_codes", "v_scales")}


def _plain_append(s):
    _plain_store(s, s["k"], s["k_codes"], s["k_scales"])
    _plain_store(s, s["v"], s["v_codes"], s["v_scales"])
    return _cache_out(s)


def _gathered(s, name):
    """Keys or values of every sequence in order, binary32 [sequences, heads, tokens, dim]."""
    table = s["page_table"].long().clamp(min=0)
    codes, e = s[name + "_codes"][table], s[name + "_scales"][table].int() - 127
    b, p, h, _, d = codes.shape
    x = codes.view(torch.float8_e4m3fn).float().view(b, p, h, PER_PAGE, BLOCK, d)
    return torch.ldexp(x, e[..., None, None]).permute(0, 2, 1, 3, 4, 5).reshape(b, h, p * PAGE, d)


def _plain_attend(s):
    c = s["case"]
    b, n, h, d = c["sequences"], c["q_tokens"], c["kv_heads"], c["head_dim"]
    group = c["q_heads"] // h
    q = s["q"].float().view(b, n, h, group, d).permute(0, 2, 3, 1, 4).reshape(b, h, group * n, d)
    k = _gathered(s, "k")
    logits = (q @ k.transpose(-1, -2)).view(b, h, group, n, -1) * s["scale"]
    here = s["lengths"].long()[:, None] - n + torch.arange(n, device=q.device)  # position of each query
    t = torch.arange(k.shape[2], device=q.device)
    seen = t <= here[..., None]
    if c["window"]:
        seen &= t > here[..., None] - c["window"]
    logits = logits.masked_fill(~seen[:, None, None], float("-inf"))
    top = logits.amax(-1, keepdim=True)
    w = torch.exp(logits - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    total = w.sum(-1, keepdim=True)
    v = _gathered(s, "v")
    o = (w.view(b, h, group * n, -1) @ v).view(b, h, group, n, d) / torch.where(total == 0, torch.ones_like(total), total)
    out = o.permute(0, 3, 1, 2, 4).reshape(b * n, -1).to(torch.bfloat16)
    if not c["lse"]:
        return out
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(b * n, -1)
    return {"out": out, "lse": lse}


def _plain_sample(s):
    logits, temperature = s["logits"].double(), s["temperature"].double()[:, None]
    vocab = logits.shape[1]
    order = torch.sort(logits, dim=-1, descending=True, stable=True)  # ties: the lowest index first
    greedy = temperature <= 0
    w = torch.exp((order.values - order.values[:, :1]) / torch.where(greedy, torch.ones_like(temperature), temperature))
    rank = torch.arange(vocab, device=logits.device)[None]
    k = s["top_k"].long()[:, None]
    k = torch.where((k <= 0) | (k > vocab), vocab, k)
    w = torch.where(rank < torch.where(greedy, 1, k), w, torch.zeros_like(w))
    mass = torch.cumsum(w, -1)
    p = s["top_p"].double()[:, None]
    kept = (mass - w < p * mass[:, -1:]) | (p >= 1) | (rank == 0)
    kept &= w >= s["min_p"].double()[:, None]
    w = torch.zeros_like(w).scatter_(1, order.indices, torch.where(kept, w, torch.zeros_like(w)))
    mass = torch.cumsum(w, -1)
    ids = torch.searchsorted(mass, s["uniform"].double()[:, None] * mass[:, -1:], right=True).clamp(max=vocab - 1)
    return {"ids": ids[:, 0].to(torch.int32), "probability": (w.gather(1, ids) / mass[:, -1:])[:, 0].float()}


# ---------------------------------------------------------------- the package's calls

def _norm_handle(mx, s):
    """What a program makes once for a layer: the norm's descriptor."""
    if "norm" not in s:
        c = s["case"]
        s["norm"] = mx.qk_norm(c["q_heads"], c["k_heads"], c["head_dim"], s["q_weight"], s["k_weight"],
                               s["inv_freq"], c["rotary_dim"], c["interleaved"], s["eps"])
        s["q_cols"] = c["q_heads"] * c["head_dim"]
    return s["norm"], s["q_cols"]


def _cache_handle(mx, s):
    if "cache" not in s:
        c = s["case"]
        s["cache"] = mx.kv_cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["pages"], PAGE,
                                 c["kv_heads"], c["head_dim"])
    return s["cache"]


def _own_rotate(mx, s):
    c = s["case"]
    t, x, y, ld = c["tokens"], s["x"], s["y"], s["x"].shape[1]
    norm, at = _norm_handle(mx, s)
    mx.mx_qk_norm_rope_bf16(x, ld, x[:, at:], ld, t, s["positions"], norm, y, ld, y[:, at:], ld)
    y = y.view(t, -1, c["head_dim"])
    return {"q": y[:, :c["q_heads"]], "k": y[:, c["q_heads"]:]}


def _own_back(mx, s):
    c = s["case"]
    t, x, dy, dx, ld = c["tokens"], s["x"], s["dy"], s["y"], s["x"].shape[1]
    norm, at = _norm_handle(mx, s)
    if "workspace" not in s:
        need = mx.mx_qk_norm_rope_backward_workspace_bytes(t, norm)
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    mx.mx_qk_norm_rope_backward_bf16(x, ld, x[:, at:], ld, dy, ld, dy[:, at:], ld, t, s["positions"], norm,
                                     dx, ld, dx[:, at:], ld, s["dq_weight"], s["dk_weight"], s["workspace"])
    dx = dx.view(t, -1, c["head_dim"])
    return {"dq": dx[:, :c["q_heads"]], "dk": dx[:, c["q_heads"]:], "dq_weight": s["dq_weight"],
            "dk_weight": s["dk_weight"]}


def _own_append(mx, s):
    c = s["case"]
    ld = c["kv_heads"] * c["head_dim"]
    starts = None if c["tokens"] == c["sequences"] else s["starts"]  # (None: as many for each)
    mx.mx_kv_append_bf16(s["k"], ld, s["v"], ld, c["tokens"], starts, s["page_table"], s["page_table"].shape[1],
                         s["lengths"], c["sequences"], _cache_handle(mx, s))
    return _cache_out(s)


def _own_attend(mx, s):
    c = s["case"]
    ld = c["q_heads"] * c["head_dim"]
    cache = _cache_handle(mx, s)
    if "workspace" not in s:
        need = mx.mx_attention_workspace_bytes(c["sequences"], c["q_tokens"], c["q_heads"], cache)
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    mx.mx_attention_bf16(s["q"], ld, c["q_heads"], c["sequences"], c["q_tokens"], s["page_table"],
                         s["page_table"].shape[1], s["lengths"], cache, s["scale"], c["window"], s["out"], ld,
                         s["lse"], s["workspace"])
    return {"out": s["out"], "lse": s["lse"]} if c["lse"] else s["out"]


def _own_sample(mx, s):
    c = s["case"]
    mx.mx_sample(s["logits"], c["rows"], c["vocab"], c["vocab"],
                 mx.MX_OUT_FP32 if c["dtype"] == "fp32" else mx.MX_OUT_BF16, s["temperature"], s["top_k"],
                 s["top_p"], s["min_p"], s["uniform"], s["ids"], s["probability"])
    return {"ids": s["ids"], "probability": s["probability"]}


def run(state):
    op = state["case"]["op"]
    if own:
        import block_scaled_fp4_bf16_gb300 as mx
        return {"rotate": _own_rotate, "back": _own_back, "append": _own_append, "attend": _own_attend,
                "sample": _own_sample}[op](mx, state)
    return {"rotate": _plain_rotate, "back": _plain_back, "append": _plain_append, "attend": _plain_attend,
            "sample": _plain_sample}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    if op in ("rotate", "back"):
        n, d = c["tokens"] * (c["q_heads"] + c["k_heads"]) * c["head_dim"], c["head_dim"]
        small = 4 * c["tokens"] + 4 * d + 2 * c["rotary_dim"]
        return {"bytes": (4 if op == "rotate" else 6) * n + small + (0 if op == "rotate" else 8 * d),
                "flops": (9 if op == "rotate" else 16) * n}
    if op == "append":
        n = 2 * c["tokens"] * c["kv_heads"] * c["head_dim"]
        blocks = 2 * (c["tokens"] // BLOCK + c["sequences"]) * c["kv_heads"]
        return {"bytes": 3 * n + blocks, "flops": 2 * n}
    if op == "attend":
        # lengths are uniform between a tenth and the whole; one is whole, one empty in a larger batch
        b, n, l = c["sequences"], c["q_tokens"], c["length"]
        mean = l if b == 1 else (l + 0.55 * l * (b - 1 - (b > 4))) / b
        seen = min(mean, c["window"] + n - 1) if c["window"] else mean
        cached = b * seen * c["kv_heads"] * 2 * (c["head_dim"] + 1.0 / BLOCK)
        rows = b * n * c["q_heads"]
        return {"bytes": int(cached + 4 * rows * c["head_dim"] + (4 * rows if c["lse"] else 0)),
                "flops": int(4 * rows * (min(seen, c["window"]) if c["window"] else seen) * c["head_dim"])}
    n = c["rows"] * c["vocab"]
    return {"bytes": n * (4 if c["dtype"] == "fp32" else 2) + 28 * c["rows"], "flops": 4 * n}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_rotate(s, c):
    t, d, r = c["tokens"], c["head_dim"], c["rotary_dim"]
    back = c["op"] == "back"
    half = r // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    phase = torch.outer(s["positions"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.ones_like(phase), phase).unsqueeze(1)
    got, at = {}, 0
    for name in ("q", "k"):
        heads, w = c[name + "_heads"], s[name + "_weight"].double()
        cols = slice(at, at + heads * d)
        at += heads * d
        x = s["x"][:, cols].double().view(t, heads, d)
        norm = ((x ** 2).sum(-1, keepdim=True) / d + s["eps"]) ** -0.5
        if not back:
            y = x * norm * w
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            got[name] = y
            continue
        g = s["dy"][:, cols].double().view(t, heads, d).clone()
        z = torch.complex(g[..., first], g[..., second]) * turn.conj()
        g[..., first], g[..., second] = z.real, z.imag
        got["d" + name + "_weight"] = torch.einsum("thd,thd->d", g, x * norm)
        gw = g * w
        got["d" + name] = norm * gw - norm ** 3 * x * ((gw * x).sum(-1, keepdim=True) / d)
    return got


def _exact_e4m3(v):
    """binary64 to the nearest E4M3 value (ties to even), as numpy."""
    a = np.abs(v)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = np.exp2(e - 3)
    return np.copysign(np.rint(a / step) * step, v)


def _e4m3_values():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where(b & 127 == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


def _exact_append(s, c):
    starts, lengths, table = (s[n].cpu().numpy() for n in ("starts", "lengths", "page_table"))
    values, got = _e4m3_values(), {}
    for name in ("k", "v"):
        codes = values[s[name + "_codes"].cpu().numpy()]
        scales = s[name + "_scales"].cpu().numpy().astype(np.int64) - 127
        new = s[name].double().cpu().numpy().reshape(c["tokens"], c["kv_heads"], c["head_dim"])
        for b in range(c["sequences"]):
            row, end = int(starts[b]), int(starts[b + 1])
            pos = int(lengths[b]) - (end - row)
            while row < end:
                page, block, off = table[b, pos // PAGE], pos % PAGE // BLOCK, pos % BLOCK
                n = min(BLOCK - off, end - row)
                x = new[row:row + n].transpose(1, 0, 2)
                top = np.abs(x).max((1, 2))
                e = np.ceil(np.log2(np.where(top > 0, top, 1.0) / 448.0)).astype(np.int64)
                e -= top <= 448.0 * np.exp2(e - 1.0)
                e += top > 448.0 * np.exp2(e)
                e = np.clip(np.where(top > 0, e, -127), -127, 127)
                held = codes[page, :, block * BLOCK:block * BLOCK + off]
                if off:
                    e = np.maximum(e, scales[page, :, block])
                    held[:] = _exact_e4m3(held * np.exp2(scales[page, :, block] - e.astype(np.float64))[:, None, None])
                lo = block * BLOCK + off
                codes[page, :, lo:lo + n] = _exact_e4m3(x * np.exp2(-e.astype(np.float64))[:, None, None])
                scales[page, :, block] = e
                row, pos = row + n, pos + n
        got[name + "_codes"] = torch.from_numpy(codes)
        got[name + "_scales"] = torch.from_numpy(np.exp2(scales.astype(np.float64)))
    return got


def _exact_attend(s, c):
    b, n, h, d = c["sequences"], c["q_tokens"], c["kv_heads"], c["head_dim"]
    group = c["q_heads"] // h
    values = torch.from_numpy(_e4m3_values()).cuda()
    q = s["q"].double().view(b, n, h, group, d)
    out = torch.zeros_like(q)
    lse = torch.full((b, n, h, group), float("-inf"), dtype=torch.float64, device="cuda")
    for i in range(b):
        length = int(s["lengths"][i])
        if not length:
            continue
        pages = s["page_table"][i, :-(-length // PAGE)].long()
        kv = []
        for name in ("k", "v"):
            x = values[s[name + "_codes"][pages].long()]
            f = torch.exp2(s[name + "_scales"][pages].double() - 127).repeat_interleave(BLOCK, -1)
            kv.append((x * f[..., None]).transpose(0, 1).flatten(1, 2)[:, :length])
        for j in range(n):
            end = length - n + j + 1
            begin = max(0, end - c["window"]) if c["window"] else 0
            if end <= 0:
                continue
            logits = s["scale"] * torch.einsum("hgd,htd->hgt", q[i, j], kv[0][:, begin:end])
            lse[i, j] = torch.logsumexp(logits, -1)
            out[i, j] = torch.einsum("hgt,htd->hgd", torch.softmax(logits, -1), kv[1][:, begin:end])
    out = out.view(b * n, -1)
    return {"out": out, "lse": lse.view(b * n, -1)} if c["lse"] else out


def _exact_sample(s, c):
    logits = s["logits"].double().cpu().numpy()
    par = {n: s[n].double().cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p", "uniform")}
    ids, prob = np.empty(c["rows"], dtype=np.int32), np.empty(c["rows"])
    for r in range(c["rows"]):
        order = np.argsort(-logits[r], kind="stable")
        if par["temperature"][r] <= 0:
            ids[r], prob[r] = order[0], 1.0
            continue
        v = logits[r, order]
        w = np.exp((v - v[0]) / par["temperature"][r])
        if 0 < par["top_k"][r] < len(w):
            w[int(par["top_k"][r]):] = 0.0
        n = len(w)
        if par["top_p"][r] < 1:
            n = max(1, int(np.searchsorted(np.cumsum(w), par["top_p"][r] * w.sum())) + 1)
        w[n:] = 0.0
        w[w < par["min_p"][r]] = 0.0
        kept = np.zeros_like(w)
        kept[order] = w
        mass = np.cumsum(kept)
        ids[r] = min(int(np.searchsorted(mass, par["uniform"][r] * mass[-1], side="right")), len(w) - 1)
        prob[r] = kept[ids[r]] / mass[-1]
    return {"ids": torch.from_numpy(ids), "probability": torch.from_numpy(prob)}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("rotate", "back"):
        return _exact_rotate(s, case)
    if op == "append":
        return _exact_append(s, case)
    return _exact_attend(s, case) if op == "attend" else _exact_sample(s, case)
