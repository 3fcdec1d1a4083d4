"""Pins of the MXFP4 oracle: the code table, ties, saturation, the scale rule,
a hand-worked block, exact round trips, non-finite blocks."""

import numpy as np
import pytest

from oracle import mxfp4_oracle as X4


def test_code_table():
    want = [0, .5, 1, 1.5, 2, 3, 4, 6]
    assert X4.e2m1_decode(np.arange(8)).tolist() == want
    assert X4.e2m1_decode(np.arange(8, 16)).tolist() == [-v for v in want]
    # the definition: bias 1, one mantissa bit, a subnormal half
    for c in range(8):
        e, m = c >> 1, c & 1
        assert want[c] == (0.5 * m if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))


@pytest.mark.parametrize("v,code", [
    (0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6),   # ties: even code
    (0.2500001, 1), (0.7499, 1), (5.01, 7), (6.0, 7), (7.9, 7), (-0.0, 8), (-5.0, 14), (-0.1, 8)])
def test_round_to_nearest_even_and_saturation(v, code):
    assert int(X4.e2m1_encode(v)) == code


def test_grid_values_round_trip_and_neighbours():
    g = X4.LADDER
    assert X4.e2m1_encode(g).tolist() == list(range(8))
    mids = (g[1:] + g[:-1]) / 2
    assert X4.e2m1_encode(np.nextafter(mids, 10)).tolist() == list(range(1, 8))
    assert X4.e2m1_encode(np.nextafter(mids, -10)).tolist() == list(range(0, 7))


def test_hand_worked_block():
    x = np.zeros((1, 64))
    x[0, :6] = [12.0, -1.0, 1.1, 0.5, 11.0, 7.0]       # max 12: X = 3 - 2 = 1
    q, s = X4.quantize(x)
    assert s.tolist() == [[128, 0]]                    # the second block is all zeros
    # x / 2: 6, -0.5, 0.55, 0.25, 5.5, 3.5 -> 6, -0.5, 0.5, 0 (tie), 6, 4 (tie)
    assert q[0, :3].tolist() == [7 | 9 << 4, 1 | 0 << 4, 7 | 6 << 4]
    assert X4.dequantize(q, s)[0, :6].tolist() == [12.0, -1.0, 1.0, 0.0, 12.0, 8.0]


def test_error_bound_and_scale_rule():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 256)) * np.exp2(rng.integers(-30, 30, (64, 1)))
    q, s = X4.quantize(x)
    d = X4.dequantize(q, s)
    sc = np.repeat(np.exp2(s.astype(float) - 127), 32, axis=1)
    amax = np.abs(x).reshape(64, 8, 32).max(2)
    assert np.all(np.floor(np.log2(amax)) - 2 == s.astype(int) - 127)
    # half a step: 1/4 of the value in the normal range, sc / 4 below it;
    # [6, 8) x scale saturates to 6
    tol = np.maximum(np.abs(x) * 0.25, sc * 0.25) + np.maximum(np.abs(x) - 6 * sc, 0)
    assert np.all(np.abs(d - x) <= tol)
    q2, s2 = X4.quantize(d)
    assert np.array_equal(X4.dequantize(q2, s2), d)


def test_non_finite_blocks_are_nan():
    x = np.ones((2, 64))
    x[0, 3], x[1, 40] = np.inf, np.nan
    q, s = X4.quantize(x)
    assert s.tolist() == [[255, 125], [125, 255]]
    d = X4.dequantize(q, s)
    assert np.isnan(d[0, :32]).all() and (d[0, 32:] == 1).all()
    assert np.isnan(d[1, 32:]).all() and (d[1, :32] == 1).all()


def test_grouped_gemm_brute_force():
    rng = np.random.default_rng(4)
    A, B = rng.standard_normal((5, 32)), rng.standard_normal((2 * 3, 32))
    out = X4.grouped_gemm(A, [0, 2, 5], B, 3)
    for r in range(5):
        e = 0 if r < 2 else 1
        for n in range(3):
            assert abs(out[r, n] - sum(A[r, k] * B[e * 3 + n, k] for k in range(32))) < 1e-12
