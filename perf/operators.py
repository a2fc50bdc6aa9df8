"""The decode-time products with FP4 weights and BF16 activations, measured.

Three operators, one pass each:

* linear:  y = act(x W^T + bias) for a few tokens, W in MXFP4 or NVFP4;
* route:   the router of a mixture-of-experts layer: gate product, the top k
           experts of each token, their softmax weights;
* experts: the products of the chosen experts, y_t = sum_j w_tj D_e (act(G_e x_t) * U_e x_t),
           with the choice given (some slots of it empty);
* layer:   route and experts, the whole layer.

`own` chooses between the plain forms below (elementary torch operations in
binary32) and the calls of the package.  W is held as the GEMM takes it: E2M1
codes, two a byte, and scales in the 128 x 4 tile order.
"""
import numpy as np
import torch

own = False

MX, NV = "mxfp4", "nvfp4"

# E2M1: 0 .5 1 1.5 2 3 4 6, sign in bit 3; both codes of a byte at once
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E2M1 = E2M1 + [-v for v in E2M1]
EDGES = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]


def block_of(fmt):
    return 32 if fmt == MX else 16


# ---------------------------------------------------------------- cases

def linear(name, tokens, n, k, fmt, out="bf16", bias=False, gelu=False):
    c = dict(op="linear", tokens=tokens, n=n, k=k, fmt=fmt, out=out, bias=bias, gelu=gelu)
    return dict(c, name=name) if name else c


def route(name, tokens, hidden, experts, top_k, normalize, masked):
    c = dict(op="route", tokens=tokens, hidden=hidden, experts=experts, top_k=top_k,
             normalize=normalize, masked=masked)
    return dict(c, name=name) if name else c


def moe(name, op, tokens, hidden, inter, experts, top_k, fmt, act, empty=0.0):
    c = dict(op=op, tokens=tokens, hidden=hidden, inter=inter, experts=experts, top_k=top_k,
             fmt=fmt, act=act, empty=empty)
    return dict(c, name=name) if name else c


def listed():
    return [
        # an attention block's square projection, one sequence decoding: launch and latency count
        linear("linear 1x4096x4096 mx", 1, 4096, 4096, MX),
        # the MLP up-projection of the decode benchmark for one sequence
        linear("linear 1x28672x8192 nv", 1, 28672, 8192, NV),
        # its down-projection for eight sequences: the longest sums
        linear("linear 8x8192x28672 mx", 8, 8192, 28672, MX),
        # the skinny benchmark's shape, binary32 out (logits)
        linear("linear 32x8192x8192 nv fp32", 32, 8192, 8192, NV, out="fp32"),
        # odd token count, sizes that are multiples of 32 only, bias and GELU
        linear("linear 5x2080x1504 mx bias gelu", 5, 2080, 1504, MX, out="fp32", bias=True, gelu=True),
        # one token's choice among 64 experts
        route("route 1x2048 of 64", 1, 2048, 64, 8, True, False),
        # a batch of 64 sequences, 256 experts of which some are switched off
        route("route 64x8192 of 256 masked", 64, 8192, 256, 8, False, True),
        # one token through a layer of small experts
        moe("layer 1x2048x1024 of 64 mx", "layer", 1, 2048, 1024, 64, 8, MX, "silu"),
        # eight sequences, most chosen experts have one token
        moe("layer 8x4096x2048 of 64 nv", "layer", 8, 4096, 2048, 64, 4, NV, "silu"),
        # a full decode batch: every expert is read, eight tokens each
        moe("layer 64x4096x2048 of 64 mx", "layer", 64, 4096, 2048, 64, 8, MX, "silu"),
        # a padded batch (slots without an expert), odd sizes, GELU gate
        moe("experts 13x1568x544 of 20 nv", "experts", 13, 1568, 544, 20, 3, NV, "gelu", empty=0.2),
        # few large experts, one token
        moe("experts 1x8192x4096 of 8 mx", "experts", 1, 8192, 4096, 8, 2, MX, "silu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _log_32(rng, lo, hi):
    """A multiple of 32 that is no multiple of 1024: those are among the listed cases."""
    n = max(1, _log_int(rng, lo // 32, hi // 32))
    return 32 * (n - 1 if n % 32 == 0 else n)


def draw(rng):
    op = rng.choice(["linear", "linear", "route", "experts", "layer"])
    fmt = rng.choice([MX, NV])
    if op == "linear":
        tokens = _log_int(rng, 1, 32)
        n, k = _log_32(rng, 256, 28672), _log_32(rng, 256, 28672)
        while n * k > 28672 * 8192:
            n, k = _log_32(rng, 256, 28672), _log_32(rng, 256, 28672)
        return linear(None, tokens, n, k, fmt, out=rng.choice(["bf16", "fp32"]),
                      bias=rng.random() < 0.3, gelu=rng.random() < 0.3)
    tokens = _log_int(rng, 1, 64)
    hidden = _log_32(rng, 512, 8192)
    experts = _log_int(rng, 4, 256)
    top_k = min(experts, rng.randint(1, 8))
    if op == "route":
        return route(None, tokens, hidden, experts, top_k, rng.random() < 0.5, rng.random() < 0.5)
    inter = _log_32(rng, 256, 4096)
    while experts * hidden * inter > 64 * 4096 * 2048:
        experts = _log_int(rng, 4, 256)
        inter = _log_32(rng, 256, 4096)
    top_k = min(experts, top_k)
    return moe(None, op, tokens, hidden, inter, experts, top_k, fmt, rng.choice(["silu", "gelu"]),
               empty=rng.choice([0.0, 0.25]) if op == "experts" else 0.0)


# ---------------------------------------------------------------- inputs

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _tile_scales(s):
    """[rows, blocks] bytes to the 128 x 4 tile order (padding 0)."""
    rows, kb = s.shape
    rt, ct = -(-rows // 128), -(-kb // 4)
    p = torch.zeros((rt * 128, ct * 4), dtype=torch.uint8, device=s.device)
    p[:rows, :kb] = s
    return p.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _quantize(w, fmt):
    """Weights [rows, k] to packed codes, tiled scales and the tensor scale (None for MXFP4)."""
    rows, k = w.shape
    b = w.view(rows, -1, block_of(fmt))
    amax = b.abs().amax(-1)
    if fmt == MX:
        e = torch.frexp(amax).exponent - 3  # floor(log2 amax) - 2
        ts, sb = None, (e + 127).clamp(0, 254).to(torch.uint8)
        q = b * torch.ldexp(torch.ones_like(amax), -e).unsqueeze(-1)
    else:
        ts = amax.amax() / 2688.0
        s8 = (amax / (6.0 * ts)).to(torch.float8_e4m3fn)
        sb = s8.view(torch.uint8)
        q = b / (s8.float() * ts).unsqueeze(-1).clamp_min(1e-30)
    code = torch.bucketize(q.abs(), torch.tensor(EDGES, device=w.device), out_int32=True).to(torch.uint8)
    code |= (q < 0).to(torch.uint8) << 3
    code = code.view(rows, k // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), _tile_scales(sb), ts


def _weights(g, count, rows, k, fmt):
    """`count` weight matrices [rows, k], stacked; sigma as a trained layer's."""
    parts = [_quantize(_randn((rows, k), g) * (0.6 * k ** -0.5 * (1.0 + 0.5 * (e % 3))), fmt)
             for e in range(count)]
    ts = None if fmt == MX else torch.stack([p[2] for p in parts])
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]), ts


def _activations(g, tokens, k):
    """Normalised activations: unit variance with a few strong channels."""
    strong = torch.rand(k, generator=g, device="cuda") < 0.01
    return (_randn((tokens, k), g) * (1.0 + 14.0 * strong)).to(torch.bfloat16)


def prepare(case, seed):
    g = _rng(seed)
    t = case["tokens"]
    s = {"case": dict(case)}
    if case["op"] == "linear":
        s["x"] = _activations(g, t, case["k"])
        codes, scales, ts = _weights(g, 1, case["n"], case["k"], case["fmt"])
        s["w"] = (codes[0], scales[0], ts)
        s["bias"] = _randn((case["n"],), g) if case["bias"] else None
        s["y"] = torch.empty((t, case["n"]), device="cuda",
                             dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        return s
    h, e, top_k = case["hidden"], case["experts"], case["top_k"]
    s["x"] = _activations(g, t, h)
    s["ids"] = torch.empty((t, top_k), device="cuda", dtype=torch.int32)
    s["weights"] = torch.empty((t, top_k), device="cuda", dtype=torch.float32)
    s["y"] = torch.empty((t, h), device="cuda", dtype=torch.bfloat16)
    if case["op"] == "experts":
        # a choice with favoured experts, as a trained router's
        logits = _randn((t, e), g) + _randn((1, e), g)
        top = logits.topk(top_k, dim=-1)
        empty = torch.rand((t, top_k), generator=g, device="cuda") < case["empty"]
        if case["empty"] > 0:
            empty[-1] = True  # a padded sequence
        s["ids"].copy_(torch.where(empty, torch.full_like(top.indices, -1), top.indices))
        s["weights"].copy_(torch.softmax(top.values, -1))
    else:
        s["router"] = (_randn((e, h), g) * (1.5 * h ** -0.5)).to(torch.bfloat16)
        s["router_bias"] = None
        if case.get("masked"):
            off = torch.rand(e, generator=g, device="cuda") < 0.25
            s["router_bias"] = torch.where(off, torch.full((e,), float("-inf"), device="cuda"),
                                           0.1 * _randn((e,), g))
    if case["op"] != "route":
        for name, rows, k in (("gate", case["inter"], h), ("up", case["inter"], h), ("down", h, case["inter"])):
            s[name] = _weights(g, e, rows, k, case["fmt"])
    return s


# ---------------------------------------------------------------- plain forms

def _dequantize(codes, scales, ts, fmt, rows, k):
    """Stacked packed codes [c, rows, k / 2] and tiled scales to binary32 [c, rows, k]."""
    c, kb = codes.shape[0], k // block_of(fmt)
    pairs = torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], device=codes.device)
    v = pairs[codes.int()].view(c, rows, kb, -1)
    rt, ct = -(-rows // 128), -(-kb // 4)
    s = scales.view(c, rt, ct, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(c, rt * 128, ct * 4)
    s = s[:, :rows, :kb].contiguous()
    s = (s.int() << 23).view(torch.float32) if fmt == MX else s.view(torch.float8_e4m3fn).float()
    v = v * s.unsqueeze(-1)
    if fmt == NV:
        v = v * ts.view(c, 1, 1, 1)
    return v.view(c, rows, k)


def _gelu(v):
    return 0.5 * v * (1.0 + torch.erf(v * 0.5 ** 0.5))


def _act(v, name):
    return _gelu(v) if name == "gelu" else v / (1.0 + torch.exp(-v))


def _plain_linear(s):
    c = s["case"]
    codes, scales, ts = s["w"]
    w = _dequantize(codes.unsqueeze(0), scales.unsqueeze(0), ts, c["fmt"], c["n"], c["k"])[0]
    y = s["x"].float() @ w.t()
    if c["bias"]:
        y = y + s["bias"]
    if c["gelu"]:
        y = _gelu(y)
    return y.to(s["y"].dtype)


def _plain_route(s):
    c = s["case"]
    logits = s["x"].float() @ s["router"].float().t()
    if s["router_bias"] is not None:
        logits = logits + s["router_bias"]
    order = torch.sort(logits, dim=-1, descending=True, stable=True)  # ties: the lowest index first
    v, ids = order.values[:, :c["top_k"]], order.indices[:, :c["top_k"]]
    e = torch.exp(v - order.values[:, :1])
    norm = e if c.get("normalize", True) else torch.exp(logits - order.values[:, :1])
    w = e / norm.sum(-1, keepdim=True)
    none = v == float("-inf")
    return (torch.where(none, torch.full_like(ids, -1), ids).to(torch.int32),
            torch.where(none, torch.zeros_like(w), w))


def _plain_experts(s, ids, weights):
    c = s["case"]
    e, t = c["experts"], c["tokens"]
    share = torch.zeros((t, e + 1), device="cuda")  # column e: slots without an expert
    share.scatter_add_(1, torch.where(ids < 0, e, ids).long(), weights)
    share = share[:, :e]
    used = torch.zeros(e + 1, device="cuda")
    used.scatter_add_(0, torch.where(ids < 0, e, ids).long().flatten(),
                      torch.ones(ids.numel(), device="cuda"))
    sel = torch.topk(used[:e], min(e, t * c["top_k"])).indices  # every expert with a token is among these

    def matrix(name, rows, k):
        codes, scales, ts = s[name]
        return _dequantize(codes[sel], scales[sel], None if ts is None else ts[sel], c["fmt"], rows, k)

    x = s["x"].float().unsqueeze(0)
    gate = x @ matrix("gate", c["inter"], c["hidden"]).transpose(1, 2)
    up = x @ matrix("up", c["inter"], c["hidden"]).transpose(1, 2)
    z = (_act(gate, c["act"]) * up) @ matrix("down", c["hidden"], c["inter"]).transpose(1, 2)
    chosen = share[:, sel].t().unsqueeze(-1)  # [selected, tokens, 1]
    return (z * chosen).sum(0).to(torch.bfloat16)


def _plain(s):
    op = s["case"]["op"]
    if op == "linear":
        return _plain_linear(s)
    if op == "experts":
        return _plain_experts(s, s["ids"], s["weights"])
    ids, weights = _plain_route(s)
    if op == "route":
        return {"ids": ids, "weights": weights}
    return {"y": _plain_experts(s, ids, weights), "ids": ids, "weights": weights}


# ---------------------------------------------------------------- the package's calls

def _experts_handle(mx, s):
    """What a program makes once when it loads the layer: the weights' descriptor and the workspace."""
    if "moe" not in s:
        c = s["case"]
        s["moe"] = mx.moe_weights(mx.MX_FMT_MXFP4 if c["fmt"] == MX else mx.MX_FMT_NVFP4, c["experts"],
                                  c["hidden"], c["inter"], s["gate"], s["up"], s["down"],
                                  mx.MX_ACT_GELU if c["act"] == "gelu" else mx.MX_ACT_SILU)
        need = mx.mx_moe_workspace_bytes(c["tokens"], c["hidden"], c["inter"], c["top_k"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s["moe"], s["workspace"]


def _calls(s):
    import block_scaled_fp4_bf16_gb300 as mx
    c, x, y = s["case"], s["x"], s["y"] if "y" in s else None
    op, t = c["op"], c["tokens"]
    if op == "linear":
        codes, scales, ts = s["w"]
        mx.mx_linear_bf16(x, t, c["k"], c["k"], mx.MX_FMT_MXFP4 if c["fmt"] == MX else mx.MX_FMT_NVFP4,
                          codes, scales, ts, c["n"], y, c["n"],
                          mx.MX_OUT_BF16 if c["out"] == "bf16" else mx.MX_OUT_FP32,
                          s["bias"], 0.0, c["gelu"])
        return y
    h, top_k = c["hidden"], c["top_k"]
    if op == "route":
        mx.mx_moe_route_bf16(x, t, h, h, s["router"], c["experts"], s["router_bias"], top_k,
                             c["normalize"], s["ids"], s["weights"])
        return {"ids": s["ids"], "weights": s["weights"]}
    handle, workspace = _experts_handle(mx, s)
    if op == "experts":
        mx.mx_moe_experts_bf16(x, t, h, s["ids"], s["weights"], top_k, handle, y, h, workspace)
        return y
    mx.mx_moe_layer_bf16(x, t, h, s["router"], s["router_bias"], top_k, True, handle, s["ids"],
                         s["weights"], y, h, workspace)
    return {"y": y, "ids": s["ids"], "weights": s["weights"]}


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def _matrix_bytes(rows, k, fmt):
    return rows * k // 2 + rows * (k // block_of(fmt))


def work(case):
    t = case["tokens"]
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        return {"bytes": _matrix_bytes(n, k, case["fmt"]) + 2 * t * k + t * n * (2 if case["out"] == "bf16" else 4)
                + (4 * n if case["bias"] else 0), "flops": 2 * t * n * k}
    h, e, top_k = case["hidden"], case["experts"], case["top_k"]
    total, flops = 2 * t * h + 8 * t * top_k, 0
    if case["op"] != "experts":
        total += 2 * e * h + (4 * e if case.get("masked") else 0)
        flops += 2 * t * e * h
    if case["op"] != "route":
        i, slots = case["inter"], t * top_k * (1.0 - case["empty"])
        active = e * (1.0 - (1.0 - (1.0 - case["empty"]) * top_k / e) ** t)  # experts with a token, expected
        total += active * (2 * _matrix_bytes(i, h, case["fmt"]) + _matrix_bytes(h, i, case["fmt"])) + 2 * t * h
        flops += 6 * slots * h * i
    return {"bytes": int(total), "flops": int(flops)}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_matrix(w, index, fmt, rows, k):
    codes, scales, ts = w
    codes = codes[index].to(torch.int64)
    table = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    v = torch.empty((rows, k), dtype=torch.float64, device=codes.device)
    v[:, 0::2] = table[codes & 15]
    v[:, 1::2] = table[codes >> 4]
    blk = block_of(fmt)
    r = torch.arange(rows, device=codes.device).unsqueeze(1)
    c = torch.arange(k // blk, device=codes.device).unsqueeze(0)
    at = ((r // 128) * (-(-(k // blk) // 4)) + c // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4
    byte = scales[index].to(torch.int64)[at]
    if fmt == MX:
        s = torch.exp2((byte - 127).double())
    else:
        exp, man = (byte >> 3) & 15, byte & 7
        s = torch.where(exp == 0, man.double() / 512, (8 + man).double() * torch.exp2((exp - 10).double()))
        s = s * ts[index].double()
    return v * s.repeat_interleave(blk, dim=1)


def _exact_route(s, c):
    logits = s["x"].double() @ s["router"].double().t()
    if s["router_bias"] is not None:
        logits += s["router_bias"].double()
    p = torch.softmax(logits, -1)
    l = logits.cpu().numpy()
    ids = np.empty((c["tokens"], c["top_k"]), dtype=np.int32)
    for t in range(c["tokens"]):
        ids[t] = np.lexsort((np.arange(l.shape[1]), -l[t]))[:c["top_k"]]
    chosen = p.gather(1, torch.from_numpy(ids).long().cuda())
    if c.get("normalize", True):
        chosen = chosen / chosen.sum(-1, keepdim=True)
    gone = np.isneginf(np.take_along_axis(l, ids.astype(np.int64), 1))
    ids[gone] = -1
    return torch.from_numpy(ids).cuda(), chosen


def exact(case, seed):
    s, c = prepare(case, seed), case
    x = s["x"].double()
    if c["op"] == "linear":
        codes, scales, ts = s["w"]
        y = x @ _exact_matrix((codes[None], scales[None], ts), 0, c["fmt"], c["n"], c["k"]).t()
        if c["bias"]:
            y = y + s["bias"].double()
        return y * 0.5 * torch.erfc(-y * 0.5 ** 0.5) if c["gelu"] else y
    if c["op"] == "experts":
        ids, weights = s["ids"], s["weights"].double()
    else:
        ids, weights = _exact_route(s, c)
    if c["op"] == "route":
        return {"ids": ids, "weights": weights}
    y = torch.zeros((c["tokens"], c["hidden"]), dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.flatten().tolist()) - {-1}):
        token, slot = (ids == e).nonzero(as_tuple=True)
        g = x[token] @ _exact_matrix(s["gate"], e, c["fmt"], c["inter"], c["hidden"]).t()
        u = x[token] @ _exact_matrix(s["up"], e, c["fmt"], c["inter"], c["hidden"]).t()
        a = g * 0.5 * torch.erfc(-g * 0.5 ** 0.5) if c["act"] == "gelu" else g * torch.sigmoid(g)
        z = (a * u) @ _exact_matrix(s["down"], e, c["fmt"], c["hidden"], c["inter"]).t()
        y.index_add_(0, token, z * weights[token, slot].unsqueeze(1))
    return y if c["op"] == "experts" else {"y": y, "ids": ids, "weights": weights}
