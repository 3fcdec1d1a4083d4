"""Pins of the FP8 layer path's oracle: the block quantisation against torch's own
E4M3 cast and hand-worked blocks, gradients against central differences."""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as X


def _bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).float().numpy()


@pytest.mark.parametrize("tall", [False, True])
def test_codes_are_torch_casts_of_the_exact_quotient(tall):
    rng = np.random.default_rng(1)
    x = _bf16(rng.standard_normal((256, 384)) * np.exp2(rng.integers(-30, 30, (256, 1))))
    q, s = X.quantize(x, tall)
    v = torch.from_numpy(x).reshape((2, 128, 3, 128) if tall else (256, 1, 3, 128))
    a = v.abs().amax((1, 3), keepdim=True)
    want = (v * 448.0 / a).to(torch.float8_e4m3fn).view(torch.uint8).reshape(256, 384).numpy()
    np.testing.assert_array_equal(q, want)
    np.testing.assert_array_equal(s, (a / 448.0)[:, 0, :, 0].numpy())
    # half a step of a value, or of the smallest code where that is more
    err = np.abs(X.dequantize(q, s) - x)
    sc = np.repeat(np.repeat(s.astype(float), 128 if tall else 1, 0), 128, 1)
    assert np.all(err <= np.maximum(np.abs(x) * 2.0 ** -4, sc * 2.0 ** -10) * (1 + 2.0 ** -20))


def test_hand_worked_block():
    x = np.zeros((1, 128))
    x[0, :8] = [448, -448, 17, 19, 1, 2.0 ** -10, 3 * 2.0 ** -10, -0.0]   # a = 448, scale 1
    q, s = X.quantize(x)
    # 17 ties between 16 (even code) and 18; 19 between 18 and 20 (even); 2^-10 between 0 and 2^-9
    assert list(X.e4m3_decode(q[0, :8])) == [448, -448, 16, 20, 1, 0, 2.0 ** -8, 0]
    assert s[0, 0] == 1.0 and q[0, 7] == 0x80
    q, s = X.quantize(x * 2.0 ** -20)
    assert s[0, 0] == 2.0 ** -20 and X.e4m3_decode(q[0, 2]) == 16


def test_zero_tiny_and_non_finite_blocks():
    x = np.zeros((4, 128))
    x[1, 3] = 2.0 ** -126
    x[2, 5], x[3, 7] = np.inf, np.nan
    q, s = X.quantize(x)
    assert s[0, 0] == s[1, 0] == 2.0 ** -125 and q[0].max() == 0 and X.e4m3_decode(q[1, 3]) == 0.5
    assert np.isnan(s[2:, 0]).all() and (q[2:] == 0x7F).all()


def test_product_against_loops():
    rng = np.random.default_rng(2)
    A, W = rng.standard_normal((5, 8)), rng.standard_normal((3 * 4, 8))
    out = X.grouped_product(A, [0, 2, 2, 5], W, 4)
    for r, e in enumerate([0, 0, 2, 2, 2]):
        for n in range(4):
            assert abs(out[r, n] - sum(A[r, k] * W[e * 4 + n, k] for k in range(8))) < 1e-12


def _differences(f, x, dir_, eps=1e-6):
    return (f(x + eps * dir_) - f(x - eps * dir_)) / (2 * eps)


@pytest.mark.parametrize("with_res", [False, True])
def test_norm_gradient_against_differences(with_res):
    rng = np.random.default_rng(3)
    x, res, w = rng.standard_normal((4, 24)), rng.standard_normal((4, 24)), rng.standard_normal(24)
    res = res if with_res else None
    dy, dsum = rng.standard_normal((4, 24)), rng.standard_normal((4, 24))
    v, _, r = X.rmsnorm(x, res, w, 1e-3)
    dx, dw = X.rmsnorm_bwd(dy, v, r, w, dsum)

    def loss(x_, w_):
        v_, y_, _ = X.rmsnorm(x_, res, w_, 1e-3)
        return (dy * y_).sum() + (dsum * v_).sum()

    for seed in range(5):
        d, dwv = np.random.default_rng(seed).standard_normal((4, 24)), np.random.default_rng(9 + seed).standard_normal(24)
        assert abs(_differences(lambda t: loss(t, w), x, d) - (dx * d).sum()) < 1e-7 * np.abs(dx * d).sum() + 1e-7
        assert abs(_differences(lambda t: loss(x, t), w, dwv) - (dw * dwv).sum()) < 1e-7 * np.abs(dw * dwv).sum() + 1e-7


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(4)
    dst = np.array([[3, 0], [1, -1], [2, 4]])
    yp, w, dy = rng.standard_normal((6, 8)), rng.random((3, 2)), rng.standard_normal((3, 8))
    into = rng.standard_normal((6, 8))
    dyp, dw = X.combine_bwd(dy, yp, dst, w, into)
    np.testing.assert_array_equal(dyp[5], into[5])          # a row that no slot names
    assert dw[1, 1] == 0.0
    for seed in range(5):
        d, dv = rng.standard_normal((6, 8)), rng.standard_normal((3, 2))
        g = _differences(lambda t: (dy * X.combine(t, dst, w)).sum(), yp, d)
        assert abs(g - (dyp[:5] * d[:5]).sum()) < 1e-7
        g = _differences(lambda t: (dy * X.combine(yp, dst, t)).sum(), w, dv)
        assert abs(g - (dw * dv).sum()) < 1e-7
