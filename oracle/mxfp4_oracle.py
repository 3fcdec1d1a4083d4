"""Plain CPU oracle for MXFP4 data (microscaled FP4 operands).

TEST INFRASTRUCTURE ONLY; shares no code with the CUDA path, float64 numpy.

The format is the published OCP Microscaling (MX) v1.0 one:
  - element: FP4 E2M1 (1 sign, 2 exponent bits with bias 1, 1 mantissa bit,
    one subnormal 0.5): 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives;
  - scale: E8M0 (code c means 2^(c - 127), 255 is NaN);
  - shared exponent of a block of 32: X = floor(log2 max|x|) - 2, clamped to
    the E8M0 range; an all-zero block takes the smallest scale;
  - element = x / 2^X rounded to nearest, ties to the even code, saturated.
A block that holds an infinity or a NaN takes the NaN scale and zero codes.
Two codes a byte, the even column in the low four bits.
"""

from __future__ import annotations

import numpy as np

BLOCK = 32
LADDER = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_decode(codes) -> np.ndarray:
    c = np.asarray(codes, np.int64) & 15
    return np.where(c & 8, -1.0, 1.0) * LADDER[c & 7]


def e2m1_encode(v) -> np.ndarray:
    """Nearest code of each float64 value; a tie goes to the even code; the sign
    bit is the input's."""
    v = np.asarray(v, np.float64)
    d = np.abs(np.abs(v)[..., None] - LADDER)
    best = d.min(-1, keepdims=True)
    near = d == best                       # one or two neighbours
    even = near & (np.arange(8) % 2 == 0)
    mag = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1))
    return (mag | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def quantize(x):
    """Rows x [R, K] -> (packed codes [R, K / 2] uint8, scale codes [R, K / 32] uint8)."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    xb = x.reshape(R, K // BLOCK, BLOCK)
    bad = ~np.isfinite(xb).all(axis=2)
    xb = np.where(bad[:, :, None], 0.0, xb)
    amax = np.abs(xb).max(axis=2)
    _, e = np.frexp(amax)
    X = np.clip(np.where(amax == 0.0, -127, e.astype(np.int64) - 1 - 2), -127, 127)
    codes = e2m1_encode(np.ldexp(xb, -X[:, :, None])).reshape(R, K)
    codes = np.where(np.repeat(bad, BLOCK, axis=1), 0, codes)
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    return packed, np.where(bad, 255, X + 127).astype(np.uint8)


def dequantize(packed, scales) -> np.ndarray:
    packed = np.asarray(packed)
    R, half = packed.shape
    v = np.empty((R, 2 * half))
    v[:, 0::2] = e2m1_decode(packed & 15)
    v[:, 1::2] = e2m1_decode(packed >> 4)
    s = np.asarray(scales, np.int64)
    v = np.ldexp(v.reshape(R, -1, BLOCK), (s - 127)[:, :, None])
    return np.where((s == 255)[:, :, None], np.nan, v).reshape(R, 2 * half)


def grouped_gemm(A, offsets, B, Nb: int) -> np.ndarray:
    """out[r] = A[r] B_e^T for the rows r of each expert e; A [P, K], B [E * Nb, K] float64."""
    out = np.zeros((A.shape[0], Nb))
    for e in range(len(offsets) - 1):
        r0, r1 = int(offsets[e]), int(offsets[e + 1])
        if r1 > r0:
            out[r0:r1] = A[r0:r1] @ B[e * Nb:(e + 1) * Nb].T
    return out
