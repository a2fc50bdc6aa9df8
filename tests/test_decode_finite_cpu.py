"""Every finite scale and every finite eps of 0 or more is taken, infinities and NaN are not (no GPU)."""
import pytest

import block_scaled_fp4_bf16_gb300 as mx
from tests.test_decode_abi_cpu import (ATTENTION, BACK, ROPE, call_attention, call_back, call_rope, lib,  # noqa: F401
                                       no_gpu, passes_the_checks)

MOST = (2 - 2.0 ** -23) * 2.0 ** 127


@no_gpu
@pytest.mark.parametrize("scale", [MOST, -MOST, 3.2e38, -3.1e38, 2.0 ** -149])
def test_scales(lib, scale):  # noqa: F811
    assert passes_the_checks(call_attention(lib)({**ATTENTION, "scale": scale})), mx.mx_last_error_string()


@no_gpu
@pytest.mark.parametrize("eps", [MOST, 3.2e38, 0.0, 2.0 ** -149])
def test_eps(lib, eps):  # noqa: F811
    for call, args in ((call_rope(lib), ROPE), (call_back(lib), BACK)):
        assert passes_the_checks(call({**args, "eps": eps})), mx.mx_last_error_string()


@pytest.mark.parametrize("v", [float("inf"), float("-inf"), float("nan")])
def test_others(lib, v):  # noqa: F811
    assert call_attention(lib)({**ATTENTION, "scale": v}) == mx.MX_ERR_INVALID_ARG
    assert call_rope(lib)({**ROPE, "eps": v}) == mx.MX_ERR_INVALID_ARG
