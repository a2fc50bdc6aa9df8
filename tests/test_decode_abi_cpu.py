"""Argument checks of the decoding step's calls (no GPU needed: they come before the device)."""
import ctypes

import pytest

import block_scaled_fp4_bf16_gb300 as mx
from block_scaled_fp4_bf16_gb300 import build as _build

MB = 1 << 20
FAKE = 0x7F0000000000
INVALID, SHAPE, ALIGN, FEATURE, WS = (mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED_SHAPE, mx.MX_ERR_ALIGNMENT,
                                      mx.MX_ERR_UNSUPPORTED_FEATURE, mx.MX_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mx.lib()


def codes_of(fn, ok, changes):
    """Each change to the valid arguments gives its status code, with a detail; the valid ones
    come as far as the device (there is none here, or the pointers would not do)."""
    for kw, want in changes:
        a = dict(ok)
        a.update(kw)
        got = fn(a)
        assert got == want, f"{kw}: {got} ({mx.mx_last_error_string()})"
        assert "no error" not in mx.mx_last_error_string()


def passes_the_checks(rc):
    return rc in (mx.MX_ERR_CUDA, mx.MX_ERR_UNSUPPORTED_ARCH, mx.MX_ERR_NOT_COMPILED)


no_gpu = pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="made-up pointers")

# q and k are columns of one row of 12 heads of 64, ld 768
NORM = dict(qh=8, kh=4, d=64, rot=64, inter=0, eps=1e-6, qw=FAKE + 4 * MB, kw=FAKE + 5 * MB, f=FAKE + 6 * MB)
ROPE = dict(NORM, q=FAKE, ldq=768, k=FAKE + 1024, ldk=768, t=10, pos=FAKE + 7 * MB, qo=FAKE + MB, ldqo=768,
            ko=FAKE + MB + 1024, ldko=768)


def norm_of(a):
    return mx.mx_qk_norm(a["qh"], a["kh"], a["d"], a["rot"], a["inter"], a["eps"], a["qw"], a["kw"], a["f"])


NORM_REFUSALS = [
    (dict(qh=0, kh=0, q=None, k=None), SHAPE), (dict(qh=-1), SHAPE), (dict(kh=65536), SHAPE),
    (dict(d=8), SHAPE), (dict(d=72), SHAPE), (dict(d=272), SHAPE), (dict(rot=8), SHAPE), (dict(rot=80), SHAPE),
    (dict(rot=-16), SHAPE), (dict(inter=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(f=None), INVALID), (dict(rot=0), INVALID), (dict(qw=FAKE + 8), ALIGN),
    (dict(kw=FAKE + 2), ALIGN), (dict(f=FAKE + 6 * MB + 2), ALIGN), (dict(t=-1), SHAPE), (dict(t=1 << 31), SHAPE),
    (dict(pos=None), INVALID), (dict(pos=FAKE + 1), ALIGN), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(kh=0), INVALID), (dict(qh=0), INVALID),                     # a pointer without heads
    (dict(ldq=511), INVALID), (dict(ldk=248), INVALID), (dict(ldq=1 << 31), INVALID), (dict(ldq=772), ALIGN),
    (dict(q=FAKE + 8), ALIGN), (dict(k=FAKE + 1026), ALIGN)]


def call_rope(lib):
    return lambda a: lib.mx_qk_norm_rope_bf16(a["q"], a["ldq"], a["k"], a["ldk"], a["t"], a["pos"],
                                              None if a.get("null") else ctypes.byref(norm_of(a)), a["qo"], a["ldqo"],
                                              a["ko"], a["ldko"], None)


def test_rope(lib):
    codes_of(call_rope(lib), ROPE, NORM_REFUSALS + [
        (dict(null=True), INVALID), (dict(qo=None), INVALID), (dict(ko=None), INVALID), (dict(ldqo=504), INVALID),
        (dict(ldko=252), INVALID), (dict(qo=FAKE + MB + 8), ALIGN), (dict(ldko=770), ALIGN),
        (dict(qo=FAKE + 16), INVALID),                               # q_out over q, shifted
        (dict(qo=FAKE, ldqo=512), INVALID),                          # at q, of another stride
        (dict(qo=FAKE + 1024), INVALID),                             # q_out over k
        (dict(ko=FAKE), INVALID),                                    # k_out over q
        (dict(ko=FAKE + MB + 1008), INVALID),                        # k_out over q_out's last head
        (dict(ko=FAKE + MB + 1280), INVALID),                        # k_out over the next row of q_out
        (dict(qo=FAKE + 4 * MB - 1024), INVALID),                    # over a weight
        (dict(qo=FAKE + 6 * MB), INVALID), (dict(ko=FAKE + 7 * MB), INVALID)])


@no_gpu
def test_rope_takes_rows_in_each_others_gaps_and_in_place(lib):
    call = call_rope(lib)
    for kw in (dict(), dict(qo=FAKE, ko=FAKE + 1024), dict(qo=FAKE), dict(kh=0, k=None, ko=None), dict(qh=0, q=None, qo=None),
               dict(ko=FAKE + 10 * 1536 + 2048), dict(qw=None, kw=None), dict(rot=0, f=None), dict(t=0)):
        assert passes_the_checks(call({**ROPE, **kw})), (kw, mx.mx_last_error_string())


BACK = dict(ROPE, dqo=FAKE + 2 * MB, lddqo=768, dko=FAKE + 2 * MB + 1024, lddko=768, dwq=FAKE + 8 * MB, dwk=FAKE + 9 * MB,
            ws=FAKE + 10 * MB, wsb=MB)


def call_back(lib):
    return lambda a: lib.mx_qk_norm_rope_backward_bf16(
        a["q"], a["ldq"], a["k"], a["ldk"], a["dqo"], a["lddqo"], a["dko"], a["lddko"], a["t"], a["pos"],
        None if a.get("null") else ctypes.byref(norm_of(a)), a["qo"], a["ldqo"], a["ko"], a["ldko"], a["dwq"], a["dwk"],
        a["ws"], a["wsb"], None)


def test_rope_backward(lib):
    need = lib.mx_qk_norm_rope_backward_workspace_bytes(10, ctypes.byref(norm_of(ROPE)))
    assert 0 < need <= MB
    codes_of(call_back(lib), BACK, NORM_REFUSALS + [
        (dict(null=True), INVALID), (dict(dqo=None), INVALID), (dict(dko=None), INVALID), (dict(lddqo=256), INVALID),
        (dict(dko=FAKE + 2 * MB + 4), ALIGN), (dict(qw=None), INVALID), (dict(kw=None), INVALID),
        (dict(dwq=FAKE + 8 * MB + 2), ALIGN), (dict(dwk=FAKE + 9 * MB + 1), ALIGN), (dict(ws=None), WS),
        (dict(wsb=need - 1), WS), (dict(ws=FAKE + 10 * MB + 8), ALIGN),
        (dict(qo=FAKE), INVALID), (dict(qo=FAKE + 2 * MB), INVALID),  # not in place
        (dict(dwq=FAKE + 2 * MB), INVALID), (dict(dwq=FAKE + 9 * MB + 64), INVALID), (dict(dwk=FAKE + MB), INVALID),
        (dict(ws=FAKE + 2 * MB), INVALID), (dict(ws=FAKE + 4 * MB), INVALID), (dict(dwq=FAKE + 10 * MB), INVALID)])


@no_gpu
def test_rope_backward_without_weights(lib):
    call = call_back(lib)
    for kw in (dict(), dict(dwq=None, dwk=None, ws=None, wsb=0), dict(dwk=None), dict(qw=None, dwq=None),
               dict(kh=0, k=None, dko=None, ko=None)):
        assert passes_the_checks(call({**BACK, **kw})), (kw, mx.mx_last_error_string())


def test_sizes_of_nothing(lib):
    n = norm_of(dict(ROPE, d=17))
    assert lib.mx_qk_norm_rope_backward_workspace_bytes(10, ctypes.byref(n)) == 0
    assert lib.mx_qk_norm_rope_backward_workspace_bytes(10, None) == 0
    assert lib.mx_qk_norm_rope_backward_workspace_bytes(-1, ctypes.byref(norm_of(ROPE))) == 0
    c = cache_of(CACHE)
    assert lib.mx_attention_workspace_bytes(4, 1, 8, ctypes.byref(c)) > 0
    for b, n, h in ((-1, 1, 8), (4097, 1, 8), (4, 0, 8), (4, 17, 8), (4, 1, 7), (4, 1, 0), (4, 1, 2 * 65)):
        assert lib.mx_attention_workspace_bytes(b, n, h, ctypes.byref(c)) == 0
    assert lib.mx_attention_workspace_bytes(4, 1, 8, None) == 0


CACHE = dict(kc=FAKE + 32 * MB, ks=FAKE + 40 * MB, vc=FAKE + 48 * MB, vs=FAKE + 56 * MB, pages=16, page=64, kvh=2, dim=128)
CALL = dict(CACHE, table=FAKE + 57 * MB, most=8, len=FAKE + 58 * MB, b=4)
CACHE_REFUSALS = [
    (dict(kc=None), INVALID), (dict(ks=None), INVALID), (dict(vc=None), INVALID), (dict(vs=None), INVALID),
    (dict(kc=FAKE + 32 * MB + 8), ALIGN), (dict(vs=FAKE + 56 * MB + 4), ALIGN), (dict(pages=0), SHAPE),
    (dict(pages=1 << 31), SHAPE), (dict(page=16), SHAPE), (dict(page=48), SHAPE), (dict(page=(1 << 20) + 32), SHAPE),
    (dict(kvh=0), SHAPE), (dict(kvh=1025), SHAPE), (dict(dim=96), SHAPE), (dict(dim=512), SHAPE), (dict(nocache=True), INVALID),
    (dict(table=None), INVALID), (dict(len=None), INVALID), (dict(table=FAKE + 2), ALIGN), (dict(len=FAKE + 1), ALIGN),
    (dict(b=-1), SHAPE), (dict(most=0), SHAPE), (dict(most=(1 << 24) + 1), SHAPE)]


def cache_of(a):
    return mx.mx_kv_cache(a["kc"], a["ks"], a["vc"], a["vs"], a["pages"], a["page"], a["kvh"], a["dim"])


def test_a_cache_past_any_memory_is_refused(lib):
    huge = dict(pages=(1 << 10) + 1, page=1 << 20, kvh=1024, dim=256)  # 2^48 codes and more: sizes stay in 64 bits
    most = dict(pages=(1 << 31) - 1, page=1 << 20, kvh=1024, dim=256)
    for a in (huge, most):
        assert call_append(lib)({**APPEND, **a, "ldk": 1 << 18, "ldv": 1 << 18}) == SHAPE
        assert call_attention(lib)({**ATTENTION, **a, "h": 1024, "ldq": 1 << 18, "ldo": 1 << 18}) == SHAPE
        assert lib.mx_attention_workspace_bytes(4, 1, 1024, ctypes.byref(cache_of({**CACHE, **a}))) == 0
    assert lib.mx_attention_workspace_bytes(4, 1, 1024, ctypes.byref(cache_of({**CACHE, **huge, "pages": 1 << 10}))) > 0


APPEND = dict(CALL, k=FAKE, ldk=256, v=FAKE + MB, ldv=256, t=8, starts=FAKE + 2 * MB)


def call_append(lib):
    return lambda a: lib.mx_kv_append_bf16(a["k"], a["ldk"], a["v"], a["ldv"], a["t"], a["starts"], a["table"], a["most"],
                                           a["len"], a["b"], None if a.get("nocache") else ctypes.byref(cache_of(a)), None)


def test_append(lib):
    codes_of(call_append(lib), APPEND, CACHE_REFUSALS + [
        (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ldk=248), INVALID), (dict(ldv=260), ALIGN),
        (dict(k=FAKE + 8), ALIGN), (dict(t=-1), SHAPE), (dict(t=(1 << 30) + 1), SHAPE), (dict(b=65536), SHAPE),
        (dict(starts=None, t=9), SHAPE), (dict(starts=FAKE + 2 * MB + 2), ALIGN),
        (dict(k=FAKE + 32 * MB), INVALID), (dict(v=FAKE + 40 * MB), INVALID), (dict(table=FAKE + 48 * MB), INVALID),
        (dict(len=FAKE + 56 * MB), INVALID), (dict(starts=FAKE + 32 * MB + 64), INVALID),
        (dict(vc=FAKE + 32 * MB), INVALID), (dict(ks=FAKE + 32 * MB + 1024), INVALID)])


@no_gpu
def test_append_allows(lib):
    for kw in (dict(), dict(starts=None), dict(t=0), dict(b=0, t=0), dict(k=FAKE, v=FAKE)):
        assert passes_the_checks(call_append(lib)({**APPEND, **kw})), (kw, mx.mx_last_error_string())


ATTENTION = dict(CALL, q=FAKE, ldq=1024, h=8, n=2, scale=0.1, window=0, o=FAKE + MB, ldo=1024, lse=FAKE + 2 * MB,
                 ws=FAKE + 64 * MB, wsb=64 * MB)


def call_attention(lib):
    return lambda a: lib.mx_attention_bf16(a["q"], a["ldq"], a["h"], a["b"], a["n"], a["table"], a["most"], a["len"],
                                           None if a.get("nocache") else ctypes.byref(cache_of(a)), a["scale"], a["window"],
                                           a["o"], a["ldo"], a["lse"], a["ws"], a["wsb"], None)


def test_attention(lib):
    need = lib.mx_attention_workspace_bytes(4, 2, 8, ctypes.byref(cache_of(CACHE)))
    assert 0 < need <= 64 * MB
    codes_of(call_attention(lib), ATTENTION, CACHE_REFUSALS + [
        (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(ldq=1016), INVALID), (dict(ldo=1028), ALIGN),
        (dict(q=FAKE + 2), ALIGN), (dict(o=FAKE + MB + 8), ALIGN), (dict(lse=FAKE + 2 * MB + 2), ALIGN),
        (dict(h=7), SHAPE), (dict(h=0), SHAPE), (dict(h=2 * 65, ldq=2 * 65 * 128), SHAPE), (dict(n=0), SHAPE),
        (dict(n=17), SHAPE), (dict(b=4097), SHAPE), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
        (dict(window=-1), INVALID), (dict(window=1 << 31), INVALID), (dict(ws=None), WS), (dict(wsb=need - 1), WS),
        (dict(ws=FAKE + 64 * MB + 8), ALIGN),
        (dict(o=FAKE), INVALID), (dict(o=FAKE + 32 * MB), INVALID), (dict(o=FAKE + 57 * MB), INVALID),
        (dict(o=FAKE + 64 * MB), INVALID), (dict(lse=FAKE + MB), INVALID), (dict(lse=FAKE), INVALID),
        (dict(lse=FAKE + 40 * MB), INVALID), (dict(ws=FAKE + 32 * MB), INVALID), (dict(ws=FAKE), INVALID)])


@no_gpu
def test_attention_allows(lib):
    for kw in (dict(), dict(lse=None), dict(b=0), dict(scale=0.0), dict(window=(1 << 31) - 1), dict(h=2)):
        assert passes_the_checks(call_attention(lib)({**ATTENTION, **kw})), (kw, mx.mx_last_error_string())


SAMPLE = dict(x=FAKE, r=4, v=1000, ld=1000, dt=1, t=FAKE + MB, k=FAKE + 2 * MB, p=FAKE + 3 * MB, m=FAKE + 4 * MB,
              u=FAKE + 5 * MB, ids=FAKE + 6 * MB, prob=FAKE + 7 * MB)


def call_sample(lib):
    return lambda a: lib.mx_sample(a["x"], a["r"], a["v"], a["ld"], a["dt"], a["t"], a["k"], a["p"], a["m"], a["u"], a["ids"],
                                   a["prob"], None)


def test_sample(lib):
    codes_of(call_sample(lib), SAMPLE, [
        (dict(x=None), INVALID), (dict(u=None), INVALID), (dict(ids=None), INVALID), (dict(dt=2), FEATURE), (dict(r=-1), SHAPE),
        (dict(r=(1 << 20) + 1), SHAPE), (dict(v=0), SHAPE), (dict(v=262145, ld=262145), SHAPE), (dict(ld=999), INVALID),
        (dict(x=FAKE + 4), ALIGN)] + [(dict([(n, FAKE + 9 * MB + 2)]), ALIGN) for n in ("t", "k", "p", "m", "u", "ids", "prob")] + [
        (dict(ids=FAKE + 4000), INVALID), (dict(prob=FAKE + 6 * MB + 12), INVALID), (dict(ids=FAKE + MB), INVALID),
        (dict(prob=FAKE + 5 * MB), INVALID)])


@no_gpu
def test_sample_allows(lib):
    for kw in (dict(), dict(t=None, k=None, p=None, m=None, prob=None), dict(r=0), dict(ld=1001, dt=0)):
        assert passes_the_checks(call_sample(lib)({**SAMPLE, **kw})), (kw, mx.mx_last_error_string())


def test_a_size_leaves_the_detail_of_the_last_call(lib):
    assert call_sample(lib)({**SAMPLE, "v": 0}) == SHAPE
    detail = mx.mx_last_error_string()
    lib.mx_attention_workspace_bytes(-1, 1, 8, ctypes.byref(cache_of(CACHE)))
    lib.mx_qk_norm_rope_backward_workspace_bytes(-1, None)
    assert mx.mx_last_error_string() == detail and "vocab" in detail


def test_descriptors_keep_their_tensors():
    import torch
    w, f = torch.ones(64, dtype=torch.bfloat16), torch.ones(16)
    n = mx.qk_norm(8, 4, 64, w, None, f)
    assert n.rotary_dim == 32 and n.q_weight == w.data_ptr() and n.k_weight is None and n.tensors[2] is f
    assert mx.qk_norm(8, 4, 64, None, None, None).rotary_dim == 0
    t = [torch.zeros(1, dtype=torch.uint8) for _ in range(4)]
    c = mx.kv_cache(*t, 1, 32, 1, 64)
    assert c.k_scales == t[1].data_ptr() and c.tensors[3] is t[3]
