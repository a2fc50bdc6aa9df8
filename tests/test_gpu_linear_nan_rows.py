"""Outputs of which some rows are NaN, for tokens that fill one, two and four loads of a
warp's sums: the NaN rows take their lanes through the sum of non-finite terms, and the
others keep their values."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
import oracle
from tests.gpu_helpers import dev_u8
from tests.test_gpu_few_tokens import FMTS, MX, assert_close, ulp, x_bits
from tests.test_gpu_linear_workspace import Wide, pick, reference, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [2, 12, 20, 32])
@pytest.mark.parametrize("n,k", [(8224, 8224), (1056, 27872)])
def test_nan_scales_of_some_rows(fmt, tokens, n, k):
    w, bits = Wide(n, k, fmt, 301), x_bits(tokens, k, 302)
    if mx.mx_linear_workspace_bytes(tokens, k, n, fmt) == 0:
        pytest.skip("a size without a workspace")
    ref, tol = reference(bits, w)
    s, bad = w.s.copy(), np.r_[np.arange(5, n, 97), n - 1]
    s[bad, (bad * 7) % s.shape[1]] = 255 if fmt == MX else 0x7F
    w.scales = dev_u8(oracle.scale_tile(s))
    for out_fp32 in (True, False):
        got = run(bits, w, out_fp32)
        want = torch.zeros(n, dtype=torch.bool)
        want[torch.from_numpy(bad)] = True
        assert torch.equal(got.isnan().cpu(), want[None].expand(tokens, n))
        fine = ~np.isin(w.rows, bad)
        assert_close(pick(got, w)[:, fine], ref[:, fine], (tol + (0 if out_fp32 else ulp(ref)))[:, fine], "rows")
