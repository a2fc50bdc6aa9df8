"""Argument checks of the few-token products (no GPU needed: they come before the device)."""
import ctypes

import pytest

import block_scaled_fp4_bf16_gb300 as mx
from block_scaled_fp4_bf16_gb300 import build as _build

MB = 1 << 20
FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return mx.lib()


def codes_of(fn, ok, changes):
    """Each change to the valid arguments gives its status code; nothing raises."""
    for kw, want in changes:
        a = dict(ok)
        a.update(kw)
        got = fn(a)
        assert got == want, f"{kw}: {got} ({mx.mx_last_error_string()})"


LINEAR = dict(x=FAKE, t=4, k=256, ldx=256, fmt=0, c=FAKE + MB, s=FAKE + 2 * MB, ts=None, n=96,
              y=FAKE + 3 * MB, ldy=96, out=0, bias=FAKE + 4 * MB, beta=0.0, gelu=0)


def test_linear(lib):
    def call(a):
        ep = mx.mx_gemm_epilogue(a["bias"], a["beta"], a["gelu"])
        return lib.mx_linear_bf16(a["x"], a["t"], a["k"], a["ldx"], a["fmt"], a["c"], a["s"], a["ts"],
                                  a["n"], a["y"], a["ldy"], a["out"], ctypes.byref(ep), None)
    codes_of(call, LINEAR, [
        (dict(x=None), mx.MX_ERR_INVALID_ARG), (dict(c=None), mx.MX_ERR_INVALID_ARG),
        (dict(s=None), mx.MX_ERR_INVALID_ARG), (dict(y=None), mx.MX_ERR_INVALID_ARG),
        (dict(fmt=2), mx.MX_ERR_INVALID_ARG),
        (dict(ts=FAKE + 5 * MB), mx.MX_ERR_INVALID_ARG),            # MXFP4 has no tensor scale
        (dict(fmt=1), mx.MX_ERR_INVALID_ARG),                       # NVFP4 needs one
        (dict(fmt=1, ts=FAKE + 5 * MB + 2), mx.MX_ERR_ALIGNMENT),
        (dict(t=-1), mx.MX_ERR_UNSUPPORTED_SHAPE), (dict(t=33), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(k=0), mx.MX_ERR_UNSUPPORTED_SHAPE), (dict(k=240), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(n=0), mx.MX_ERR_UNSUPPORTED_SHAPE), (dict(n=100), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(n=1 << 31), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(n=1 << 24, k=1 << 13, ldx=1 << 13, ldy=1 << 24), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(ldx=248), mx.MX_ERR_INVALID_ARG), (dict(ldy=95), mx.MX_ERR_INVALID_ARG),
        (dict(ldx=260), mx.MX_ERR_ALIGNMENT), (dict(x=FAKE + 8), mx.MX_ERR_ALIGNMENT),
        (dict(c=FAKE + MB + 4), mx.MX_ERR_ALIGNMENT), (dict(s=FAKE + 2 * MB + 4), mx.MX_ERR_ALIGNMENT),
        (dict(y=FAKE + 3 * MB + 2), mx.MX_ERR_ALIGNMENT), (dict(bias=FAKE + 4 * MB + 4), mx.MX_ERR_ALIGNMENT),
        (dict(out=2), mx.MX_ERR_UNSUPPORTED_FEATURE), (dict(gelu=2), mx.MX_ERR_INVALID_ARG),
        (dict(y=FAKE + 16), mx.MX_ERR_INVALID_ARG),                 # y over x
        (dict(y=FAKE + MB + 4096), mx.MX_ERR_INVALID_ARG),          # y over the codes
        (dict(y=FAKE + 2 * MB), mx.MX_ERR_INVALID_ARG),             # y over the scales
        (dict(y=FAKE + 4 * MB - 16), mx.MX_ERR_INVALID_ARG),        # y over the bias
    ])


ROUTE = dict(x=FAKE, t=4, h=256, ldx=256, r=FAKE + MB, e=16, b=FAKE + 2 * MB, k=4, norm=1,
             ids=FAKE + 3 * MB, w=FAKE + 4 * MB)


def test_route(lib):
    def call(a):
        return lib.mx_moe_route_bf16(a["x"], a["t"], a["h"], a["ldx"], a["r"], a["e"], a["b"], a["k"],
                                     a["norm"], a["ids"], a["w"], None)
    codes_of(call, ROUTE, [
        (dict(x=None), mx.MX_ERR_INVALID_ARG), (dict(r=None), mx.MX_ERR_INVALID_ARG),
        (dict(ids=None), mx.MX_ERR_INVALID_ARG), (dict(w=None), mx.MX_ERR_INVALID_ARG),
        (dict(norm=2), mx.MX_ERR_INVALID_ARG),
        (dict(t=65), mx.MX_ERR_UNSUPPORTED_SHAPE), (dict(h=48, ldx=48), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(e=0), mx.MX_ERR_UNSUPPORTED_SHAPE), (dict(e=513), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(k=0), mx.MX_ERR_UNSUPPORTED_SHAPE), (dict(k=17, e=64), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(e=3), mx.MX_ERR_UNSUPPORTED_SHAPE),                   # top_k above the experts
        (dict(ldx=128), mx.MX_ERR_INVALID_ARG), (dict(ldx=260), mx.MX_ERR_ALIGNMENT),
        (dict(r=FAKE + MB + 8), mx.MX_ERR_ALIGNMENT), (dict(b=FAKE + 2 * MB + 2), mx.MX_ERR_ALIGNMENT),
        (dict(ids=FAKE + 3 * MB + 1), mx.MX_ERR_ALIGNMENT),
        (dict(w=FAKE + 3 * MB + 32), mx.MX_ERR_INVALID_ARG),        # weights over ids
        (dict(ids=FAKE + 64), mx.MX_ERR_INVALID_ARG),               # ids over x
    ])


def _moe(fmt=0, act=0, e=8, h=256, i=128, ts=(None, None, None), base=FAKE + 8 * MB, **kw):
    m = [(base + j * 4 * MB, base + j * 4 * MB + 2 * MB, ts[j]) for j in range(3)]
    for name, v in kw.items():
        j, f = int(name[1]), int(name[3])
        m[j] = m[j][:f] + (v,) + m[j][f + 1:]
    return mx.moe_weights(fmt, e, h, i, *m, act)


EXPERTS = dict(x=FAKE, t=4, ldx=256, ids=FAKE + MB, w=FAKE + 2 * MB, k=2, m={}, y=FAKE + 3 * MB, ldy=256,
               ws=FAKE + 4 * MB, wsb=MB)


def test_workspace_bytes(lib):
    assert mx.mx_moe_workspace_bytes(4, 256, 128, 2) >= 4 * 2 * (256 + 128) * 4
    for bad in ((0, 256, 128, 2), (65, 256, 128, 2), (4, 0, 128, 2), (4, 256, -1, 2), (4, 256, 128, 0),
                (4, 256, 128, 17)):
        assert mx.mx_moe_workspace_bytes(*bad) == 0


def test_experts_and_layer(lib):
    def experts(a):
        moe = None if a["m"] is None else ctypes.byref(_moe(**a["m"]))
        return lib.mx_moe_experts_bf16(a["x"], a["t"], a["ldx"], a["ids"], a["w"], a["k"], moe, a["y"],
                                       a["ldy"], a["ws"], a["wsb"], None)

    def layer(a):
        moe = None if a["m"] is None else ctypes.byref(_moe(**a["m"]))
        return lib.mx_moe_layer_bf16(a["x"], a["t"], a["ldx"], a.get("r", FAKE + 6 * MB), a.get("b"), a["k"],
                                     a.get("norm", 1), moe, a["ids"], a["w"], a["y"], a["ldy"], a["ws"],
                                     a["wsb"], None)
    ts = FAKE + 7 * MB
    changes = [
        (dict(x=None), mx.MX_ERR_INVALID_ARG), (dict(m=None), mx.MX_ERR_INVALID_ARG),
        (dict(ids=None), mx.MX_ERR_INVALID_ARG), (dict(w=None), mx.MX_ERR_INVALID_ARG),
        (dict(y=None), mx.MX_ERR_INVALID_ARG), (dict(m=dict(fmt=3)), mx.MX_ERR_INVALID_ARG),
        (dict(m=dict(act=2)), mx.MX_ERR_INVALID_ARG), (dict(m=dict(m0f0=None)), mx.MX_ERR_INVALID_ARG),
        (dict(m=dict(m1f1=None)), mx.MX_ERR_INVALID_ARG), (dict(m=dict(m2f2=ts)), mx.MX_ERR_INVALID_ARG),
        (dict(m=dict(fmt=1, ts=(ts, None, ts))), mx.MX_ERR_INVALID_ARG),
        (dict(m=dict(fmt=1, ts=(ts, ts, ts + 2))), mx.MX_ERR_ALIGNMENT),
        (dict(m=dict(m2f0=FAKE + 8 * MB + 8)), mx.MX_ERR_ALIGNMENT),
        (dict(t=65), mx.MX_ERR_UNSUPPORTED_SHAPE), (dict(k=0), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(k=17), mx.MX_ERR_UNSUPPORTED_SHAPE), (dict(m=dict(e=0)), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(m=dict(e=513)), mx.MX_ERR_UNSUPPORTED_SHAPE), (dict(m=dict(i=48)), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(m=dict(h=272), ldx=272, ldy=272), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(ldx=248), mx.MX_ERR_INVALID_ARG), (dict(ldy=255), mx.MX_ERR_INVALID_ARG),
        (dict(ldx=257), mx.MX_ERR_ALIGNMENT), (dict(y=FAKE + 3 * MB + 8), mx.MX_ERR_ALIGNMENT),
        (dict(ids=FAKE + MB + 2), mx.MX_ERR_ALIGNMENT),
        (dict(ws=None), mx.MX_ERR_WORKSPACE), (dict(wsb=1024), mx.MX_ERR_WORKSPACE),
        (dict(ws=FAKE + 4 * MB + 4), mx.MX_ERR_ALIGNMENT),
        (dict(y=FAKE + 64), mx.MX_ERR_INVALID_ARG),                        # y over x
        (dict(y=FAKE + 4 * MB), mx.MX_ERR_INVALID_ARG),                    # y over the workspace
        (dict(ws=FAKE + 8 * MB), mx.MX_ERR_INVALID_ARG),                   # workspace over the gate codes
        (dict(y=FAKE + 16 * MB), mx.MX_ERR_INVALID_ARG),                   # y over the down codes
        (dict(ws=FAKE + 2 * MB), mx.MX_ERR_INVALID_ARG),                   # workspace over the weights
    ]
    codes_of(experts, EXPERTS, changes)
    codes_of(layer, EXPERTS, changes)
    codes_of(layer, EXPERTS, [
        (dict(r=None), mx.MX_ERR_INVALID_ARG), (dict(norm=-1), mx.MX_ERR_INVALID_ARG),
        (dict(m=dict(e=1)), mx.MX_ERR_UNSUPPORTED_SHAPE),                  # top_k above the experts
        (dict(ids=FAKE + 6 * MB), mx.MX_ERR_INVALID_ARG),                  # ids over the router
        (dict(ids=FAKE + 8 * MB), mx.MX_ERR_INVALID_ARG),                  # ids over the gate codes
        (dict(y=FAKE + 6 * MB + 64), mx.MX_ERR_INVALID_ARG),               # y over the router
        (dict(b=FAKE + 4 * MB), mx.MX_ERR_INVALID_ARG),                    # the bias in the workspace
    ])


def test_linear_workspace(lib):
    """A size that takes a workspace: its refusals, and those of the plain call."""
    ok = dict(LINEAR, k=8192, ldx=8192, n=28672, ldy=28672, x=FAKE, c=FAKE + 256 * MB, s=FAKE + 512 * MB,
              y=FAKE + 16 * MB, bias=FAKE + 32 * MB, ws=FAKE + 64 * MB, wsb=None)
    need = mx.mx_linear_workspace_bytes(4, 8192, 28672, 0)
    assert need > 0

    def call(a):
        ep = mx.mx_gemm_epilogue(a["bias"], a["beta"], a["gelu"])
        return lib.mx_linear_bf16_workspace(
            a["x"], a["t"], a["k"], a["ldx"], a["fmt"], a["c"], a["s"], a["ts"], a["n"], a["y"], a["ldy"],
            a["out"], ctypes.byref(ep), a["ws"], need if a["wsb"] is None else a["wsb"], None)
    codes_of(call, ok, [
        (dict(ws=None), mx.MX_ERR_WORKSPACE), (dict(wsb=need - 1), mx.MX_ERR_WORKSPACE),
        (dict(ws=FAKE + 64 * MB + 8), mx.MX_ERR_ALIGNMENT),
        (dict(ws=FAKE + 256 * MB), mx.MX_ERR_INVALID_ARG),          # over the codes
        (dict(ws=FAKE), mx.MX_ERR_INVALID_ARG),                     # over x
        (dict(ws=FAKE + 16 * MB), mx.MX_ERR_INVALID_ARG),           # over y
        (dict(x=None), mx.MX_ERR_INVALID_ARG), (dict(t=33), mx.MX_ERR_UNSUPPORTED_SHAPE),
        (dict(k=8200), mx.MX_ERR_UNSUPPORTED_SHAPE), (dict(fmt=3), mx.MX_ERR_INVALID_ARG),
        (dict(out=2), mx.MX_ERR_UNSUPPORTED_FEATURE),
    ])


def test_messages_name_the_call(lib):
    lib.mx_linear_bf16(None, 1, 32, 32, 0, None, None, None, 32, None, 32, 0, None, None)
    assert "mx_linear_bf16" in mx.mx_last_error_string() and "x is null" in mx.mx_last_error_string()
