"""min_p above 1: the first of the largest logits is kept, alone, whatever ties with it or weighs as
much to the weights' accuracy."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests.gpu_helpers import check_guards, guarded
from tests.test_gpu_sample import normal

pytestmark = pytest.mark.gpu


def sample(x, bf16, uniform, **parameters):
    rows, vocab = x.shape
    t = torch.from_numpy(x).to("cuda", torch.bfloat16 if bf16 else torch.float32)
    ids, prob = guarded(rows, torch.int32, 77), guarded(rows, torch.float32, 7.0)
    par = {k: torch.full((rows,), v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda")
           for k, v in parameters.items()}
    u = torch.tensor(uniform, dtype=torch.float32, device="cuda")
    mx.mx_sample(t, rows, vocab, vocab, mx.MX_OUT_BF16 if bf16 else mx.MX_OUT_FP32, par.get("temperature"), par.get("top_k"),
                 par.get("top_p"), par.get("min_p"), u, ids, prob)
    assert mx.mx_device_status() == 0
    check_guards(ids, prob)
    return ids.tolist(), prob.tolist()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab", [10, 5003, 151937])
@pytest.mark.parametrize("min_p", [1 + 2.0 ** -23, 7.0, 3e38, np.inf])
def test_above_one(vocab, min_p, bf16):
    x = np.minimum(normal(5, vocab, seed=vocab), 1.5)
    at = sorted({vocab // 3, vocab // 2, vocab - 1})
    x[:2, at] = 5.0
    x[2, 1], x[2, at[1]] = 2.0 - 2.0 ** -7, 2.0  # (as much to the weights' accuracy at a high temperature)
    x[3, at] = np.inf
    x[4] = -np.inf
    u = [0.9, 0.0, 0.999, 0.9, 0.5]
    for extra in ({}, {"top_k": 2, "top_p": 0.9}, {"temperature": 1e30}, {"temperature": 0.0}):
        ids, prob = sample(x, bf16, u, min_p=min_p, **extra)
        assert ids == [at[0], at[0], at[1], at[0], -1]
        assert prob == [1.0, 1.0, 1.0, 1.0, 0.0]


@pytest.mark.parametrize("bf16", [False, True])
def test_one_keeps_what_ties(bf16):
    x = np.minimum(normal(3, 5003, seed=1), 1.5)
    x[:, [11, 4000]] = 5.0
    ids, prob = sample(x, bf16, [0.2, 0.7, 0.99], min_p=1.0)
    assert ids == [11, 4000, 4000] and prob == [0.5] * 3
