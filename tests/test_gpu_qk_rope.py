"""mx_qk_norm_rope_bf16 and its gradients against the formulas in binary64.

Tolerances: a norm's factor, a sine or cosine and the products with them are a dozen binary32
roundings of 2^-24 and an angle exact to 2^-32 of a turn, so a rotated pair (a, b) is off by at
most 2^-19 (|a| + |b|), a gradient by 2^-18 of the sum of its terms' magnitudes (its mean adds up
to 256 products); BF16 outputs by half a step, 2^-8 relative, more.  Weight gradients are sums of
up to `terms` products in binary32: (2^-18 + terms 2^-24) of their magnitudes."""
import numpy as np
import pytest
import torch

import block_scaled_fp4_bf16_gb300 as mx
from tests import decode_ref as ref
from tests.gpu_helpers import check_guards, guarded

pytestmark = pytest.mark.gpu


class Case:
    """Queries and keys as columns of one wider row, outputs between guards."""

    def __init__(self, tokens, q_heads, k_heads, dim, rotary, interleaved, seed=0, weights=(True, True),
                 positions=None, pad=8, eps=1e-6):
        rng = np.random.default_rng(seed)
        self.t, self.heads, self.dim, self.pad = tokens, (q_heads, k_heads), dim, pad
        self.ld = (q_heads + k_heads) * dim + 2 * pad
        self.x = ref.bf16_round(rng.normal(size=(tokens, self.ld)) * np.exp(rng.normal(size=(tokens, 1))))
        self.dy = ref.bf16_round(rng.normal(size=(tokens, self.ld)))
        self.w = [ref.bf16_round(1 + 0.3 * rng.normal(size=dim)) if on else None for on in weights]
        self.f = (10000.0 ** (-np.arange(rotary // 2) / max(1, rotary // 2))).astype(np.float32)
        self.pos = rng.integers(0, 100000, tokens) if positions is None else np.resize(positions, tokens)
        self.rotary, self.interleaved, self.eps = rotary, interleaved, eps
        dev = lambda v, t=torch.bfloat16: None if v is None else torch.from_numpy(np.asarray(v)).to("cuda", t)  # noqa: E731
        self.dev = dev
        self.inv_freq = dev(self.f, torch.float32) if rotary else None
        self.positions = dev(self.pos, torch.int32)
        self.norm = mx.qk_norm(q_heads, k_heads, dim, dev(self.w[0]), dev(self.w[1]), self.inv_freq, rotary,
                               interleaved, eps)

    def cols(self, part):
        at = self.pad + part * (self.heads[0] * self.dim + self.pad // 8 * 8)
        return slice(at, at + self.heads[part] * self.dim)

    def of(self, rows, part):
        return rows[:, self.cols(part)].reshape(self.t, self.heads[part], self.dim)

    def view(self, rows, part):
        return rows[:, self.cols(part)] if self.heads[part] else None

    def buffer(self):
        body = guarded(self.t * self.ld, torch.bfloat16, 3.0)
        out = body.view(self.t, self.ld)
        out._mx_guard = body._mx_guard
        return out

    def untouched(self, out, what=3.0):
        mask = np.ones(self.ld, bool)
        for part in range(2):
            mask[self.cols(part)] = False
        assert (out.double().cpu().numpy()[:, mask] == what).all()

    def args(self, part):
        return (self.w[part], self.eps, self.pos, self.f, self.rotary, self.interleaved)

    def forward(self, x, out):
        mx.mx_qk_norm_rope_bf16(self.view(x, 0), self.ld, self.view(x, 1), self.ld, self.t, self.positions,
                                self.norm, self.view(out, 0), self.ld, self.view(out, 1), self.ld)

    def check_forward(self, out):
        got = out.double().cpu().numpy()
        for part in range(2):
            x = self.of(self.x, part)
            want = ref.norm_rotate(x, *self.args(part))
            size = ref.rotate_size(ref.norm_rotate(x, self.w[part], self.eps, self.pos, self.f, 0, False),
                                   self.rotary, self.interleaved)
            err = np.abs(self.of(got, part) - want)
            assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size).all(), (part, err.max())


SHAPES = [  # tokens, q_heads, k_heads, dim, rotary
    (1, 1, 1, 16, 16), (1, 32, 8, 128, 128), (3, 5, 2, 32, 16), (5, 7, 1, 48, 48), (37, 12, 4, 64, 32), (2, 3, 3, 80, 64),
    (9, 4, 0, 96, 96), (9, 0, 3, 112, 16), (4, 3, 1, 192, 128), (3, 9, 2, 256, 256), (3, 9, 2, 144, 0), (700, 40, 9, 128, 64)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, interleaved):
    c = Case(*shape, interleaved, seed=sum(shape))
    out = c.buffer()
    c.forward(c.dev(c.x), out)
    c.check_forward(out)
    c.untouched(out)
    check_guards(out)


@pytest.mark.parametrize("weights", [(False, False), (True, False), (False, True)])
def test_forward_without_norms(weights):
    c = Case(6, 5, 3, 64, 64, False, weights=weights)
    out = c.buffer()
    c.forward(c.dev(c.x), out)
    c.check_forward(out)


@pytest.mark.parametrize("interleaved", [False, True])
def test_forward_in_place(interleaved):
    c = Case(70, 6, 2, 128, 96, interleaved)
    x = c.dev(c.x)
    c.forward(x, x)
    c.check_forward(x)


@pytest.mark.parametrize("position", [0, 1, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -1, -(2 ** 31)])
def test_far_positions(position):
    c = Case(2, 2, 1, 128, 128, False, positions=[position])
    out = c.buffer()
    c.forward(c.dev(c.x), out)
    c.check_forward(out)


def test_frequencies_of_any_size():
    c = Case(4, 2, 1, 64, 64, True, positions=[3, 1001, 77777, -5])
    c.f = np.array([65536.0, 1000.5, -3.25, 0.0, 1e-30, 2.0 ** -140] + [2.0 ** -i for i in range(26)], np.float32)
    c.inv_freq.copy_(torch.from_numpy(c.f))
    out = c.buffer()
    c.forward(c.dev(c.x), out)
    # (2^16 * 77777 is 2^32 radians: the definition's own angle is exact to 2^-21)
    got = out.double().cpu().numpy()
    for part in range(2):
        want = ref.norm_rotate(c.of(c.x, part), *c.args(part))
        assert (np.abs(c.of(got, part) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15).all()


def test_infinities_and_nan_stay_in_their_head():
    c = Case(5, 4, 2, 64, 64, False)
    clean = c.buffer()
    c.forward(c.dev(c.x), clean)
    x = c.x.copy()
    x[1, c.cols(0).start + 64 + 3] = np.inf     # token 1, query head 1
    x[3, c.cols(1).start + 5] = np.nan          # token 3, key head 0
    out = c.buffer()
    c.forward(c.dev(x), out)
    same = (out == clean).cpu().numpy()
    bad = np.zeros_like(same)
    bad[1, c.cols(0).start + 64:c.cols(0).start + 128] = True
    bad[3, c.cols(1).start:c.cols(1).start + 64] = True
    assert same[~bad].all()
    assert torch.isnan(out[3, c.cols(1).start:c.cols(1).start + 64]).all()


def test_zero_rows_and_no_tokens():
    c = Case(3, 2, 1, 64, 32, False)
    c.x[:] = 0
    out = c.buffer()
    c.forward(c.dev(c.x), out)
    c.check_forward(out)
    mx.mx_qk_norm_rope_bf16(out, c.ld, out[:, 128:], c.ld, 0, c.positions, c.norm, out, c.ld, out[:, 128:], c.ld)


def backward(c, x, dy, dx, weights=(True, True)):
    dw = [guarded(c.dim, torch.float32, 7.0) if on and c.w[p] is not None else None for p, on in enumerate(weights)]
    need = mx.mx_qk_norm_rope_backward_workspace_bytes(c.t, c.norm)
    ws = guarded(need)
    mx.mx_qk_norm_rope_backward_bf16(c.view(x, 0), c.ld, c.view(x, 1), c.ld, c.view(dy, 0), c.ld, c.view(dy, 1), c.ld,
                                     c.t, c.positions, c.norm, c.view(dx, 0), c.ld, c.view(dx, 1), c.ld, dw[0], dw[1], ws)
    torch.cuda.synchronize()
    check_guards(dx, dw[0], dw[1], ws)
    return dw


def check_backward(c, dx, dw):
    got = dx.double().cpu().numpy()
    for part in range(2):
        want, want_w, size, size_w = ref.norm_rotate_backward(c.of(c.x, part), c.of(c.dy, part), *c.args(part))
        err = np.abs(c.of(got, part) - want)
        assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size).all(), (part, err.max())
        if dw[part] is not None:
            terms = c.t * c.heads[part]
            err = np.abs(dw[part].double().cpu().numpy() - want_w)
            assert (err <= (2.0 ** -18 + terms * 2.0 ** -24) * size_w).all(), (part, err.max())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, interleaved):
    c = Case(*shape, interleaved, seed=1 + sum(shape))
    dx = c.buffer()
    dw = backward(c, c.dev(c.x), c.dev(c.dy), dx)
    check_backward(c, dx, dw)
    c.untouched(dx)


@pytest.mark.parametrize("weights", [(False, False), (True, False), (False, True)])
def test_backward_without_norms(weights):
    c = Case(6, 5, 3, 64, 64, False, weights=weights)
    dx = c.buffer()
    check_backward(c, dx, backward(c, c.dev(c.x), c.dev(c.dy), dx))


def test_backward_without_weight_gradients():
    c = Case(6, 5, 3, 64, 64, False)
    dx = c.buffer()
    check_backward(c, dx, backward(c, c.dev(c.x), c.dev(c.dy), dx, (False, False)))
    check_backward(c, dx, backward(c, c.dev(c.x), c.dev(c.dy), dx, (False, True)))


def test_backward_gives_the_same_bits_again():
    c = Case(900, 10, 3, 128, 128, False)
    x, dy, one, two = c.dev(c.x), c.dev(c.dy), c.buffer(), c.buffer()
    a, b = backward(c, x, dy, one), backward(c, x, dy, two)
    assert torch.equal(one, two) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim, rotary", [(80, 80), (144, 64), (48, 0)])
def test_backward_does_not_see_the_weights_of_a_call_before(dim, rotary, interleaved):
    """A head of 5 x 16 channels leaves lanes without any: what another call left on chip stays out."""
    c, last = Case(3000, 3, 2, dim, rotary, interleaved), Case(3000, 2, 2, 256, 256, interleaved)
    bad = torch.full((256,), np.inf, dtype=torch.bfloat16, device="cuda")
    last.norm = mx.qk_norm(2, 2, 256, bad, bad, last.inv_freq, 256, interleaved)
    x, dy, dx = c.dev(c.x), c.dev(c.dy), c.buffer()
    last_x, last_dx = last.dev(last.x), last.buffer()
    backward(last, last_x, last_x, last_dx)
    check_backward(c, dx, backward(c, x, dy, dx))


def test_backward_of_no_tokens_clears_the_weights_gradients():
    c = Case(3, 2, 1, 64, 64, False)
    c.t = 0
    x = c.dev(c.x)
    dw = [torch.full((64,), 7.0, device="cuda") for _ in range(2)]
    ws = torch.empty(mx.mx_qk_norm_rope_backward_workspace_bytes(0, c.norm), dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(x)
    mx.mx_qk_norm_rope_backward_bf16(x, c.ld, x[:, 128:], c.ld, x, c.ld, x[:, 128:], c.ld, 0, c.positions, c.norm, dx,
                                     c.ld, dx[:, 128:], c.ld, dw[0], dw[1], ws)
    assert (dw[0] == 0).all() and (dw[1] == 0).all()


def test_gradients_agree_with_differences_of_the_forward_call():
    """Along a direction: the forward call's change and the gradients' prediction of it."""
    c = Case(4, 3, 2, 64, 64, False, positions=[5])
    dx = c.buffer()
    backward(c, c.dev(c.x), c.dev(c.dy), dx)
    rng = np.random.default_rng(9)
    step = 2.0 ** -4
    way = rng.choice([-1.0, 1.0], size=c.x.shape) * np.abs(c.x) * step  # BF16 sums stay close to exact
    up, down = ref.bf16_round(c.x + way), ref.bf16_round(c.x - way)
    a, b = c.buffer(), c.buffer()
    c.forward(c.dev(up), a)
    c.forward(c.dev(down), b)
    for part in range(2):
        got = (c.of(c.dy, part) * (c.of(a.double().cpu().numpy(), part) - c.of(b.double().cpu().numpy(), part))).sum()
        delta = c.of(up - down, part)
        want = (c.of(dx.double().cpu().numpy(), part) * delta).sum()
        # outputs' rounding (2^-8 each, random signs: a standard deviation of their root sum, times 5), second order:
        # a cubic term of step^2 relative to the change of the terms
        size = ref.rotate_size(ref.norm_rotate(c.of(c.x, part), *c.args(part)), 64, False)
        noise = 5 * 2.0 ** -8 * np.sqrt(2 * (c.of(c.dy, part) ** 2 * size ** 2).sum())
        assert abs(got - want) <= noise + 4 * step ** 2 * (np.abs(c.of(dx.double().cpu().numpy(), part)) * np.abs(delta)).sum()
