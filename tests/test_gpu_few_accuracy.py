"""How near moe_layer_fwd_few and moe_layer_fwd_few_mxfp4 come to the float64
oracle where the ordinary tokens of test_gpu_few.py cannot tell.

The bound of an element is that of test_gpu_few.py, from the absolute values of
the same products, with what E2M1 parts leave as PARTS of a block's largest value
or 2^-129, whichever is more: the scales end at 2^-127, and a last part there
rounds to steps of 1/2."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu
from oracle import moe_oracle as O
from oracle import mxfp4_oracle as X4
from test_gpu_few import U, Few, bf16

pytestmark = [pytest.mark.gpu, needs_gpu]

PARTS = 2.0 ** -11   # four parts


def left(v):
    """What the parts of each block of 32 leave, at most."""
    m = np.abs(v).reshape(len(v), -1, 32).max(2)
    return np.repeat(np.maximum(PARTS * m, 2.0 ** -129), 32, axis=1)


class Case(Few):
    """SwiGLU experts without biases."""

    def expert(self, x, w1, w2, b1, b2):
        F, h = self.F, self.h
        z = x @ w1.T
        dz = h * U * (np.abs(x) @ np.abs(w1).T)
        if self.mx:
            dz = dz + left(x) @ np.abs(w1).T
        g, u, dg, du = z[:, :F], z[:, F:], dz[:, :F], dz[:, F:]
        a = O.silu(g) * u
        da = 1.13 * dg * (np.abs(u) + du) + (np.abs(O.silu(g)) + 1.13 * dg) * du
        da = da + 2.0 ** -18 * (np.abs(a) + da)
        many = self.T > 8 and self.T * self.K > 4 * self.E
        da = da + (left(np.abs(a) + da) if self.mx else 2.0 ** (-8 if many else -16) * (np.abs(a) + da))
        return a @ w2.T, da @ np.abs(w2).T + F * U * (np.abs(a) @ np.abs(w2).T)

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
