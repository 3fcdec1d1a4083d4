"""Plain CPU oracle of the FP8 layer path: block-of-128 quantisation, the grouped
products, the RMS norm and its gradient, the combine's gradient.

TEST INFRASTRUCTURE ONLY; shares no code with the CUDA path, float64 numpy.

A block (1 x 128 of activations, 128 x 128 of weights) whose largest magnitude
is m has a = max(m, 448 2^-125), the scale fp32(a / 448) and the codes
E4M3(448 x / a), to nearest with ties to the even code.  A block that holds an
infinity or a NaN has a NaN scale and the codes 0x7F.
"""

from __future__ import annotations

import numpy as np

from .mxfp8_oracle import e4m3_decode, e4m3_encode, silu

BLOCK, TOP = 128, 448.0
FLOOR = TOP * 2.0 ** -125


def _blocks(x, tall):
    R, K = x.shape
    rb = BLOCK if tall else 1
    return x.reshape(R // rb, rb, K // BLOCK, BLOCK)


def quantize(x, tall=False):
    """x [R, K] -> (codes [R, K] uint8, scales [R or R / 128, K / 128] float32)."""
    x = np.asarray(x, np.float64)
    b = _blocks(x, tall)
    bad = ~np.isfinite(b).all(axis=(1, 3))
    b = np.where(bad[:, None, :, None], 0.0, b)
    a = np.maximum(np.abs(b).max(axis=(1, 3)), FLOOR)
    codes = e4m3_encode(b * TOP / a[:, None, :, None])
    codes = np.where(bad[:, None, :, None], 0x7F, codes).astype(np.uint8)
    scales = np.where(bad, np.float32(np.nan), a.astype(np.float32) / np.float32(TOP))
    return codes.reshape(x.shape), scales.astype(np.float32)


def dequantize(codes, scales):
    """float64 values of codes [R, K]; scales [R, K / 128] or [R / 128, K / 128]."""
    v = e4m3_decode(codes)
    s = np.asarray(scales, np.float64)
    s = np.repeat(np.repeat(s, v.shape[0] // s.shape[0], axis=0), BLOCK, axis=1)
    return v * s


def grouped_product(A, offsets, W, Nw):
    """out[r] = A[r] W_e^T for the rows r of each expert; W [E * Nw, K]."""
    out = np.zeros((A.shape[0], Nw))
    for e in range(len(offsets) - 1):
        r0, r1 = int(offsets[e]), int(offsets[e + 1])
        if r1 > r0:
            out[r0:r1] = A[r0:r1] @ W[e * Nw:(e + 1) * Nw].T
    return out


def swiglu(H, p):
    F = H.shape[1] // 2
    return np.asarray(p, np.float64)[:, None] * silu(H[:, :F]) * H[:, F:]


def rmsnorm(x, res, w, eps):
    """(v, y, r): v = x + res, r = (mean v^2 + eps)^(-1/2), y = v r w."""
    v = np.asarray(x, np.float64) + (0.0 if res is None else np.asarray(res, np.float64))
    r = 1.0 / np.sqrt((v * v).mean(axis=1) + eps)
    return v, v * r[:, None] * np.asarray(w, np.float64), r


def rmsnorm_bwd(dy, v, r, w, dsum=None):
    """(dx, dw) from the forward's v and r."""
    dy, v, w = (np.asarray(t, np.float64) for t in (dy, v, w))
    n = v * np.asarray(r, np.float64)[:, None]
    g = dy * w
    dx = np.asarray(r, np.float64)[:, None] * (g - n * (g * n).mean(axis=1, keepdims=True))
    return dx if dsum is None else dx + np.asarray(dsum, np.float64), (dy * n).sum(axis=0)


def combine(y_perm, dst_row, w):
    """y[t] = sum_k w[t, k] y_perm[dst_row[t, k]]; rows -1 add nothing."""
    dst = np.asarray(dst_row)
    rows = np.asarray(y_perm, np.float64)[np.maximum(dst, 0)]
    return (np.where(dst >= 0, w, 0.0)[:, :, None] * rows).sum(axis=1)


def combine_bwd(dy, y_perm, dst_row, w, into):
    """(dy_perm, dw); rows of dy_perm that no slot names are those of `into`."""
    dy, dst = np.asarray(dy, np.float64), np.asarray(dst_row)
    out = np.array(into, np.float64)
    dw = np.zeros(dst.shape)
    for t, k in zip(*np.nonzero(dst >= 0)):
        out[dst[t, k]] = w[t, k] * dy[t]
        dw[t, k] = dy[t] @ np.asarray(y_perm[dst[t, k]], np.float64)
    return out, dw
