"""The decoding step's 64-bit definitions against differences, brute force and known values."""
import numpy as np
import pytest
import torch

from tests import decode_ref as ref


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [0, 16, 32])
@pytest.mark.parametrize("weighted", [False, True])
def test_gradients_are_those_of_differences(interleaved, rotary, weighted):
    rng = np.random.default_rng(5)
    x, dy = rng.normal(size=(3, 2, 32)), rng.normal(size=(3, 2, 32))
    w = rng.normal(size=32) if weighted else None
    f, pos = 10.0 ** -np.arange(rotary // 2), np.array([0, 7, -123456])

    def loss(x, w):
        return (ref.norm_rotate(x, w, 1e-3, pos, f, rotary, interleaved) * dy).sum()

    dx, dw, _, _ = ref.norm_rotate_backward(x, dy, w, 1e-3, pos, f, rotary, interleaved)
    step = 1e-6
    for at in [(0, 0, 0), (1, 1, 5), (2, 0, 17), (2, 1, 31)]:
        e = np.zeros_like(x)
        e[at] = step
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - dx[at]) < 1e-7
    if weighted:
        for d in (0, 9, 31):
            e = np.zeros(32)
            e[d] = step
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * step) - dw[d]) < 1e-7


def test_e4m3_rounding_is_torchs():
    v = torch.cat([torch.linspace(-448, 448, 20001, dtype=torch.float64),
                   torch.logspace(-11, 2, 5001, base=2.0, dtype=torch.float64)]).float()
    want = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_round(v.double().numpy()), want)
    assert np.array_equal(ref.e4m3_round(np.array([np.inf, -np.inf, np.nan, 0.0, -0.0])), [0x7F, 0x7F, 0x7F, 0, 0x80])
    bytes_ = torch.arange(256, dtype=torch.uint8)
    table = bytes_.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(table), np.isnan(ref.E4M3))
    assert np.array_equal(np.nan_to_num(table), np.nan_to_num(ref.E4M3))


def test_tokens_one_by_one_are_the_tokens_together_where_scales_do_not_grow():
    rng = np.random.default_rng(1)
    x = ref.bf16_round(rng.normal(size=(70, 2, 64)))
    x[:, :, 0] = 4.0  # every block's scale is that of its first token
    x = np.clip(x, -4, 4)
    a, b = (ref.Cache(4, 64, 2, 64, [[2, 0]], 3) for _ in range(2))
    a.append((x, -x), [70], [70])
    for i in range(70):
        b.append((x[i:i + 1], -x[i:i + 1]), [1], [i + 1])
    for w in range(2):
        va, vb = a.values(w, 0, 70)[0], b.values(w, 0, 70)[0]
        assert np.array_equal(va, vb)


def test_sampling_follows_its_definition():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    got = [ref.sample(l, 1.0, 0, 1.0, 0.0, u)[0] for u in (0.0, 0.05, 0.11, 0.45, 0.55, 0.75, 0.99)]
    assert got == [0, 0, 1, 1, 2, 3, 3]
    assert [ref.sample(l, 1.0, 2, 1.0, 0.0, u)[0] for u in (0.0, 0.55, 0.6, 0.9)] == [1, 1, 3, 3]
    assert [ref.sample(l, 1.0, 0, 0.65, 0.0, u)[0] for u in (0.0, 0.6)] == [1, 3]       # 0.4 + 0.3 >= 0.65
    assert [ref.sample(l, 1.0, 0, 1.0, 0.45, u)[0] for u in (0.0, 0.43, 0.45, 0.66, 0.67)] == [1, 1, 2, 2, 3]  # >= 0.18
    assert ref.sample(l, 0.0, 0, 1.0, 0.0, 0.9)[:2] == (1, 1.0)
    assert ref.sample(np.array([-np.inf, -np.inf]), 1.0, 0, 1.0, 0.0, 0.5)[0] == -1
