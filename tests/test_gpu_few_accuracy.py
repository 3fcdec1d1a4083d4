"""How near moe_layer_fwd_few and moe_layer_fwd_few_mxfp4 come to the float64
oracle where the ordinary tokens of test_gpu_few.py cannot tell.

The bound of an element is that of test_gpu_few.py, from the absolute values of
the same products: the hidden values beside bf16 weights are two bf16 numbers, the
second what the first (half a step, 2^-8) left, so within 2^-16, however many tokens
an expert has; what E2M1 parts leave is PARTS of a block's largest value or 2^-129,
whichever is more: the scales end at 2^-127, and a last part there rounds to steps of
1/2."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu, to_np
from oracle import moe_oracle as O
from oracle import mxfp4_oracle as X4
from test_gpu_few import U, Few, bf16

pytestmark = [pytest.mark.gpu, needs_gpu]

PARTS = 2.0 ** -17   # six parts, three bits each


def left(v):
    """What the parts of each block of 32 leave, at most."""
    m = np.abs(v).reshape(len(v), -1, 32).max(2)
    return np.repeat(np.maximum(PARTS * m, 2.0 ** -129), 32, axis=1)


class Case(Few):
    def expert(self, x, w1, w2, b1, b2):
        F, h = self.F, self.h
        z = x @ w1.T + (0 if b1 is None else b1)
        dz = h * U * (np.abs(x) @ np.abs(w1).T + (0 if b1 is None else np.abs(b1)))
        if self.mx:
            dz = dz + left(x) @ np.abs(w1).T
        if self.act == 1:
            g, u, dg, du = z[:, :F], z[:, F:], dz[:, :F], dz[:, F:]
            a = O.silu(g) * u
            da = 1.13 * dg * (np.abs(u) + du) + (np.abs(O.silu(g)) + 1.13 * dg) * du
        else:
            a, da = O.gelu(z), 1.13 * dz
        da = da + 2.0 ** -18 * (np.abs(a) + da)
        da = da + (left(np.abs(a) + da) if self.mx else 2.0 ** -16 * (np.abs(a) + da))
        o = a @ w2.T + (0 if b2 is None else b2)
        return o, da @ np.abs(w2).T + F * U * (np.abs(a) @ np.abs(w2).T)

    def exact(self):
        """y in 64 bits for the routing and the weights of it that the call returned."""
        x, y = self.x.astype(np.float64), np.zeros((self.T, self.h))
        idx, prob = to_np(self.idx).astype(int), to_np(self.prob).astype(np.float64)
        m = lambda w, e: None if w is None else w[e].astype(np.float64)  # noqa: E731
        for e in np.unique(idx):
            t, k = np.nonzero(idx == e)
            o = self.expert(x[t], m(self.w1, e), m(self.w2, e), m(self.b1, e), m(self.b2, e))[0]
            y[t] += prob[t, k][:, None] * o
        if self.shared:
            y += self.expert(x, self.w1s.astype(np.float64), self.w2s.astype(np.float64), None, None)[0]
        return y

    def set_w1(self, w1):
        """First projections with these values (to bf16, then to MXFP4 where that is used)."""
        self.w1 = bf16(w1)
        if self.mx:
            self.w1_bf16 = self.w1
            q = X4.quantize(self.w1.reshape(-1, self.h))
            self.w1 = X4.dequantize(*q).reshape(self.w1.shape)


def checked(f):
    M = lib()
    f.device(M).call(M)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    f.check(M)
    return f


def only_the_output_rounding(f):
    """The error as a whole is that of rounding y to bf16.  Steps are 2^-7 of y's power
    of two, and rounding errors spread evenly over a step, so their squares' mean is
    step^2 / 12; over n elements the norm scatters by 0.45 / sqrt(n / 2) of itself (n of
    thousands here, the steps differing in size), and 1.05 is several times that.  The
    fp32 sums and the tokens' and hidden values' representation have to vanish beside it:
    2^-16 of the hidden values is 1/150 of the bf16 rounding, hidden values of one bf16
    number make the ratio 1.4; four E2M1 parts of tokens and hidden values make it 1.15,
    six leave an error 64 times smaller."""
    y = f.exact()
    step = np.exp2(np.floor(np.log2(np.abs(y) + 1e-300)) - 7)
    err = to_np(f.y).astype(np.float64) - y
    assert y.size >= 4096
    assert np.linalg.norm(err) <= 1.05 * np.sqrt((step ** 2).sum() / 12), \
        np.linalg.norm(err) / np.sqrt((step ** 2).sum() / 12)


def ends(x_exp, w_exp, mx):
    """Tokens times 2^x_exp, first projections times 2^w_exp; routing is forced, with
    equal weights, so the logits' size does not matter."""
    f = Case(T=5, h=256, E=4, K=2, F=128, mx=mx, force=True, seed=17)
    f.w_r[:] = 0.0
    f.x = bf16(np.ldexp(f.x.astype(np.float64), x_exp))
    f.set_w1(np.ldexp(f.w1_bf16 if mx else f.w1, w_exp))
    return f


@pytest.mark.parametrize("mx", [False, True])
def test_tokens_near_the_largest_numbers(mx):
    """Blocks whose largest value is between 3.5 2^126 and 2^128: four units of
    their first scale, which a part may round to, are no fp32 number."""
    f = ends(124, -119, mx)
    f.x[1, 3::32] = bf16(3.0e38)
    f.x[2, 7::32] = bf16(-3.3e38)
    f.x[3, :] = bf16(2.99e38)
    assert np.isfinite(f.x).all() and np.abs(f.x).max() > 3.5 * 2.0 ** 126
    checked(f)


@pytest.mark.parametrize("mx", [False, True])
def test_tokens_near_the_smallest_numbers(mx):
    """Blocks whose parts' scales end at 2^-127, bf16 subnormals among them."""
    f = ends(-122, 119, mx)
    f.x[1] = bf16(np.ldexp(f.x[1].astype(np.float64), -6))
    f.x[2] = 0.0
    f.x[3, 1::2] = bf16(2.0 ** -133)
    checked(f)


FEW = [
    dict(T=8, h=1032, E=8, K=2, F=512, shared=1),
    dict(T=5, h=1024, E=256, K=8, F=136, score=1, sel=True, shared=1),
]
MANY = [  # more than four tokens an expert: units of 16 tokens
    dict(T=9, h=512, E=1, K=1, F=520),
    dict(T=16, h=1024, E=4, K=2, F=512, shared=1),
    dict(T=33, h=640, E=2, K=1, F=384),
    dict(T=64, h=512, E=1, K=1, F=256, shared=1),
    dict(T=40, h=264, E=5, K=3, F=1000, act=0, bias=True),
    dict(T=47, h=136, E=9, K=4, F=5008),
]


def _id(c):
    return f"T{c['T']}_E{c['E']}_F{c['F']}"


@pytest.mark.parametrize("c", FEW + MANY, ids=_id)
def test_bf16_weights_leave_the_output_rounding(c):
    only_the_output_rounding(checked(Case(**c)))


MX = [
    dict(T=1, h=4096, E=4, K=2, F=256),
    dict(T=5, h=1152, E=256, K=8, F=128, score=1, sel=True, shared=1),
    dict(T=8, h=1024, E=1, K=1, F=640),
    dict(T=13, h=512, E=8, K=2, F=1024, gate=True),
    dict(T=33, h=384, E=3, K=2, F=256, renorm=False),
    dict(T=64, h=256, E=2, K=2, F=512, shared=1),
]


@pytest.mark.parametrize("c", MX, ids=_id)
def test_mxfp4_weights_leave_the_output_rounding(c):
    only_the_output_rounding(checked(Case(mx=True, **c)))


@pytest.mark.parametrize("T", [6, 30])
def test_what_stands_beside_an_outlier_in_a_block(T):
    """A value of 100 in one of a token's 32 blocks, which meets zero weights: the
    result is that of the other values.  Six parts leave at most 2^-17 100 = 1/1300 of
    those beside it, 1/2300 in the mean, and as these are a 32nd of the products some
    1/10000 of a result, a fifteenth of the output rounding; four parts (2^-11 100) would
    leave four times that rounding."""
    f = Case(T=T, h=1024, E=2, K=1, F=256, mx=True)
    f.x[:, 40] = 100.0
    w1 = f.w1_bf16.copy()
    w1[:, :, 40] = 0.0
    f.set_w1(w1)
    only_the_output_rounding(checked(f))


def test_a_token_has_one_error_whatever_the_batch():
    """Eight tokens of one expert in a unit of 8, and with a ninth in a unit of 16: the
    rows differ by their fp32 sums' orders alone, some 2^-20 of the result, and that moves
    an element to the next bf16 number in about one case in 2^12 (2^-20 beside a step of
    2^-8); rounding the hidden values otherwise, by 2^-9, would move every third one."""
    nine = Case(T=9, h=512, E=1, K=1, F=384)
    checked(nine)
    eight = Case(T=8, h=512, E=1, K=1, F=384, x=nine.x[:8])
    eight.w_r, eight.w1, eight.w2 = nine.w_r, nine.w1, nine.w2
    checked(eight)
    assert (eight.y != nine.y[:8]).float().mean() < 0.02
