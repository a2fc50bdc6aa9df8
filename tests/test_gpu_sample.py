"""mx_sample against its definition in binary64: ids equal (no case's deciding border is within 2^-38
of its total, the weights' own accuracy), probabilities within 2^-22 relative (one rounding to
binary32, and 2^-38)."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests import decode_ref as ref
from tests.gpu_helpers import check_guards, guarded

pytestmark = pytest.mark.gpu


def run(logits, temperature=None, top_k=None, top_p=None, min_p=None, uniform=None, bf16=False, pad=0, probability=True):
    """logits: binary64 [rows, vocab] (rounded to the type first); parameters: one a row or None."""
    rows, vocab = logits.shape
    ld = vocab + pad
    t = torch.full((rows, ld), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    t[:, :vocab] = torch.from_numpy(np.asarray(logits)).to("cuda", t.dtype)
    dev = lambda v, d=torch.float32: None if v is None else torch.tensor(np.asarray(v), device="cuda").to(d)  # noqa: E731
    ids, prob = guarded(rows, torch.int32, 77), guarded(rows, torch.float32, 7.0)
    par = [dev(temperature), dev(top_k, torch.int32), dev(top_p), dev(min_p)]
    u = dev(uniform)
    mx.mx_sample(t, rows, vocab, ld, mx.MX_OUT_BF16 if bf16 else mx.MX_OUT_FP32, *par, u, ids, prob if probability else None)
    assert mx.mx_device_status() == 0
    check_guards(ids, prob)
    got = ids.cpu().numpy(), prob.double().cpu().numpy()
    value = t[:, :vocab].double().cpu().numpy()
    default = (1.0, 0, 1.0, 0.0)
    for r in range(rows):
        p = [default[i] if par[i] is None else par[i][r].item() for i in range(4)]
        want, w_prob, near = ref.sample(value[r], *p, u[r].item())
        assert near > 2.0 ** -38, "a case on a border"
        assert got[0][r] == want, (r, got[0][r], want, p, near)
        if probability:
            assert abs(got[1][r] - w_prob) <= 2.0 ** -22 * w_prob, (r, got[1][r], w_prob)
    return got


def normal(rows, vocab, sigma=2.5, seed=0):
    return np.random.default_rng(seed).normal(size=(rows, vocab)) * sigma


def uniforms(rows, seed=1):
    return np.random.default_rng(seed).random(rows).astype(np.float32)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 511, 513, 1000, 4096, 4097, 20011, 65536, 151937, 262144])
def test_vocabularies(vocab, bf16):
    rows = 12
    x = normal(rows, vocab, seed=vocab)
    u = uniforms(rows, vocab)
    run(x, uniform=u, bf16=bf16, pad=3)
    run(x, temperature=np.linspace(0.3, 2.0, rows), top_k=[0, 1, 2, 3, 5, 8, 20, 50, 100, 1000, vocab, vocab + 5],
        uniform=u, bf16=bf16)
    run(x, top_p=np.linspace(0.05, 0.999, rows), uniform=u, bf16=bf16)
    run(x, min_p=np.linspace(0.0, 0.9, rows) + 0.013, uniform=u, bf16=bf16)
    run(x, temperature=np.linspace(0.5, 1.5, rows), top_k=np.arange(rows) * 37 + 1, top_p=np.linspace(0.5, 1.1, rows),
        min_p=np.linspace(0, 0.2, rows), uniform=u, bf16=bf16)


def test_many_rows():
    rows = 700
    rng = np.random.default_rng(3)
    run(normal(rows, 3000, seed=4), temperature=rng.choice([0.0, 0.5, 1.0], rows), top_k=rng.choice([0, 1, 40], rows),
        top_p=rng.choice([1.0, 0.9, 0.3], rows), min_p=rng.choice([0.0, 0.05], rows), uniform=uniforms(rows))


@pytest.mark.parametrize("rows,vocab", [(100, 40001), (512, 16001), (513, 16001)])
def test_rows_that_do_not_all_run_at_once(rows, vocab):
    """Rows with top-p begin first; each row's answer stays its own."""
    rng = np.random.default_rng(rows)
    x = normal(rows, vocab, seed=rows)
    x[7, 3], x[9] = np.nan, -np.inf
    t = rng.choice([0.0, 0.6, 1.2], rows)
    t[11] = np.nan
    run(x, temperature=t, top_k=rng.choice([0, 30, 3000], rows), top_p=rng.choice([1.0, 0.9, 0.4], rows),
        min_p=rng.choice([0.0, 0.03], rows), uniform=uniforms(rows, rows))
    run(x[:, :vocab], top_p=rng.choice([1.0, 0.7], rows), uniform=uniforms(rows, rows + 1))


@pytest.mark.parametrize("uniform", [0.0, 2.0 ** -30, 0.5, 1 - 2.0 ** -24, 1.0, 2.0, -1.0])
def test_ends_of_the_uniform_numbers(uniform):
    x = np.concatenate([normal(3, 5001, seed=6), np.full((1, 5001), 0.25)])
    run(x[:3], uniform=[uniform] * 3)
    got = run(x[:3], top_k=[1, 2, 7], uniform=[uniform] * 3)
    if uniform >= 1:  # the last kept one, by index
        top = np.argsort(-x[1].astype(np.float32), kind="stable")[:2]
        assert got[0][1] == top.max()


def test_ties_go_to_the_lowest_index():
    x = np.zeros((6, 9000))
    x[:, [4000, 17, 8999, 5, 8000]] = 3.0
    top = np.array([5, 17, 4000, 8000, 8999])
    got = run(x, temperature=[0.0] * 6, uniform=[0.3] * 6)
    assert (got[0] == 5).all()
    for k in range(1, 6):  # which of the equal ones are kept
        for j in range(k):
            got = run(x[:1], top_k=[k], uniform=[(j + 0.5) / k])
            assert got[0][0] == top[j] and abs(got[1][0] - 1 / k) < 1e-6
    e = np.exp(3.0) * 5
    for n in range(1, 6):  # the fewest that reach top_p
        p = np.float32((n - 0.5) / 5 * e / (e + 8995))
        assert run(x[:1], top_p=[p], uniform=[0.999])[0][0] == top[n - 1]
    # a top-k border inside the ties, and a top-p border inside of what that keeps
    got = run(x[:1], top_k=[4], top_p=[0.7], uniform=[0.999])
    assert got[0][0] == top[2]


def test_masked_and_empty_rows():
    x = normal(8, 6000, seed=8)
    x[0, :5999] = -np.inf
    x[1] = -np.inf
    x[2, ::2] = -np.inf
    x[3, 100] = np.nan
    x[4, [7, 4500]] = np.inf
    x[5] = -3.0e38
    x[5, 10] = 3.0e38
    u = [0.9] * 8
    t = [1.0] * 6 + [np.nan, 1.0]
    got = run(x, temperature=t, uniform=u)
    assert got[0][0] == 5999 and got[0][1] == -1 and got[0][3] == -1 and got[0][4] == 4500 and got[0][5] == 10
    assert got[0][6] == -1 and got[1][1] == 0.0 and got[1][4] == 0.5
    run(x, temperature=t, top_k=[3] * 8, top_p=[0.9] * 8, min_p=[0.01] * 8, uniform=u)
    run(x, temperature=[0.0] * 8, uniform=u)
    got = run(x, top_p=[np.nan] + [0.9] * 7, min_p=[0.1] * 2 + [np.nan] + [0.1] * 5, uniform=u[:7] + [np.nan])
    assert got[0][0] == -1 and got[0][2] == -1 and got[0][7] == -1


@pytest.mark.parametrize("temperature", [1e-38, 2.0 ** -100, 1e-6, 0.01, 50.0, 1e30, -1.0])
def test_temperatures(temperature):
    x = normal(3, 4099, seed=10)
    run(x, temperature=[temperature] * 3, uniform=uniforms(3))
    run(x, temperature=[temperature] * 3, top_k=[5, 50, 500], top_p=[0.99, 0.51, 0.9311], uniform=uniforms(3))


def test_flat_and_peaked_rows():
    x = normal(4, 100003, sigma=1e-3, seed=11)
    x[2:] *= 3e4
    u = uniforms(4)
    run(x, uniform=u)
    run(x, top_p=[0.9, 0.1, 0.9, 0.999], uniform=u)
    run(x, top_k=[30000, 77777, 5, 40000], uniform=u)


def test_odd_parameters():
    x = normal(6, 2000, seed=12)
    u = uniforms(6)
    run(x, top_k=[-5, 0, 2000, 1999, 2 ** 31 - 1, 1], uniform=u)
    run(x, top_p=[0.0, -1.0, 1.0, 7.0, 2.0 ** -30, 2.0 ** -60], uniform=u, probability=False)
    run(x, min_p=[0.0, -1.0, 1.0, 7.0, 2.0 ** -43.5, 1e-30], uniform=u)


def test_the_same_bits_again_and_no_rows():
    x = torch.from_numpy(normal(40, 50000, seed=13)).float().cuda()
    u = torch.rand(40, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    p = torch.full((40,), 0.95, device="cuda")
    outs = []
    for _ in range(3):
        ids, prob = torch.empty(40, dtype=torch.int32, device="cuda"), torch.empty(40, device="cuda")
        mx.mx_sample(x, 40, 50000, 50000, mx.MX_OUT_FP32, None, None, p, None, u, ids, prob)
        outs.append((ids, prob))
    assert all(torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1]) for a, b in outs)
    mx.mx_sample(x, 0, 50000, 50000, mx.MX_OUT_FP32, None, None, p, None, u, ids, prob)
