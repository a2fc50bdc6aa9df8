"""mx_linear_bf16 is one call whichever way its stream is named: the same kernels (so the
same bits) with the stream as an argument, as a handle, and as the current one."""
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests.gpu_helpers import dev_bf16
from tests.test_gpu_few_tokens import FMTS, x_bits
from tests.test_gpu_linear_workspace import Wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,n,k", [(4, 8224, 8224), (24, 8224, 8224), (3, 96, 1056)])
def test_the_same_bits(fmt, tokens, n, k):
    w, x = Wide(n, k, fmt, 501), dev_bf16(x_bits(tokens, k, 502))

    def call(y, stream=None):
        mx.mx_linear_bf16(x, tokens, k, k, fmt, w.codes, w.scales, w.ts, n, y, n, mx.MX_OUT_FP32, stream=stream)
        return y
    new = lambda: torch.full((tokens, n), float("nan"), device="cuda")  # noqa: E731
    want, side = call(new()), torch.cuda.Stream()
    outs = [new() for _ in range(5)]
    torch.cuda.synchronize()
    call(outs[0], side)
    call(outs[1], side.cuda_stream)
    call(outs[2], 0)                 # the default stream
    call(outs[3], 1)                 # the same by its other handle
    with torch.cuda.stream(side):
        call(outs[4])
    torch.cuda.synchronize()
    assert torch.isfinite(want).all()
    for y in outs:
        assert torch.equal(y, want)


def test_workspaces_of_calls_in_flight_on_two_given_streams():
    """Calls that overlap on two streams, neither the current one."""
    t, n, k, fmt = 2, 8224, 8224, mx.MX_FMT_MXFP4
    w, xs = Wide(n, k, fmt, 511), [dev_bf16(x_bits(t, k, 512 + i)) for i in range(8)]
    new = lambda: torch.empty(t, n, device="cuda")  # noqa: E731

    def call(x, y, stream=None):
        mx.mx_linear_bf16(x, t, k, k, fmt, w.codes, w.scales, w.ts, n, y, n, mx.MX_OUT_FP32, stream=stream)
        return y
    want, streams = [call(x, new()) for x in xs], [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[new() for _ in xs] for _ in range(10)]
    torch.cuda.synchronize()
    for ys in got:
        for i, (x, y) in enumerate(zip(xs, ys)):
            call(x, y, streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(y, v) for ys in got for y, v in zip(ys, want))


def test_a_given_stream_in_a_graph():
    t, n, k, fmt = 4, 8224, 8224, mx.MX_FMT_NVFP4
    w, x, y = Wide(n, k, fmt, 521), dev_bf16(x_bits(t, k, 522)), torch.zeros(4, 8224, device="cuda")

    def call(stream=None):
        mx.mx_linear_bf16(x, t, k, k, fmt, w.codes, w.scales, w.ts, n, y, n, mx.MX_OUT_FP32, stream=stream)
    call()
    torch.cuda.synchronize()
    want, graph, side = y.clone(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call(side)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
