"""Where mx_linear_bf16 takes its workspace from when it is given none (no GPU: the library
is a stand-in that notes what it is called with)."""
import pytest
import torch

from block_scaled_fp4_bf16_gb300 import _binding as b

NEED = 4096


class Library:
    def __init__(self):
        self.calls = []

    def mx_linear_workspace_bytes(self, tokens, k, n, fmt):
        return NEED

    def mx_linear_bf16(self, *args):
        self.calls.append(("without", None, None))
        return 0

    def mx_linear_bf16_workspace(self, *args):
        self.calls.append(("with", args[13], args[14]))
        return 0


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(b, "lib", lambda: lib)
    monkeypatch.setattr(b, "_stream", lambda s: s)
    b.mx_linear_workspace_bytes.cache_clear()
    yield lib
    b.mx_linear_workspace_bytes.cache_clear()


def call(x, **kw):
    b.mx_linear_bf16(x, 1, 8192, 8192, b.MX_FMT_MXFP4, 1 << 20, 2 << 20, None, 28672, 3 << 20, 28672, **kw)


def test_no_workspace_in_host_memory(library):
    """x in host memory that the GPU reads (pinned): the workspace must not lie beside it."""
    call(torch.zeros(1, 8192, dtype=torch.bfloat16))
    assert library.calls == [("without", None, None)]


def test_an_address_goes_without(library):
    call(1 << 24)
    assert library.calls == [("without", None, None)]


def test_a_given_workspace_is_used(library):
    ws = torch.zeros(NEED, dtype=torch.uint8)
    call(1 << 24, workspace=ws)
    call(1 << 24, workspace=1 << 25, workspace_bytes=NEED)
    assert library.calls == [("with", ws.data_ptr(), NEED), ("with", 1 << 25, NEED)]
