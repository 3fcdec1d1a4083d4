"""moe_expert_fc1_mxfp4 with strongly negative gates, where SiLU decays to nothing.

Tokens of ones and gate weights of one value make a gate z the same exact number in
every product order.  CUDA bounds __expf(-z) by 2 + |1.173 z| units in the last place
(2^-23 of the value each), __fdividef by 2, and four more roundings (the sum, the two
products, p) by half a unit each: 2^-23 (6 + 1.173 |z|) of a in all.  A quotient below
2^-126 may come out as 0: another |z u| 2^-126.  The bf16 output adds half a step: 2^-8 of
the value, or half of the smallest subnormal, 2^-134."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu, to_np
from oracle import mxfp4_oracle as X4
from test_gpu_mxfp4 import bf16, quantize_dev

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("z", [-8.0, -24.0, -48.0, -64.0, -96.0, -128.0, -768.0])
def test_strongly_negative_gates(z):
    M = lib()
    P, h, F = 40, 128, 256
    rng = np.random.default_rng(int(-z))
    w1 = np.empty((2 * F, h), np.float32)
    w1[:F] = z / h                                   # one E2M1 value and a power of two: exact
    w1[F:] = bf16(rng.standard_normal((F, h)))
    cfg = M.make_config(P, h, 1, 1, F)
    od = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    xq, xsf = quantize_dev(M, np.ones((P, h), np.float32), 1, [0, P])
    wq, wsf = quantize_dev(M, w1, 1)
    a = torch.full((P, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    M.moe_expert_fc1_mxfp4(cfg, xq, xsf, od, None, wq, wsf, a, None, None)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    w = X4.dequantize(*X4.quantize(w1))
    assert np.all(w[:F] == z / h)
    u, du = w[F:].sum(1), h * 2.0 ** -23 * np.abs(w[F:]).sum(1)   # the up sums: as in test_gpu_mxfp4.py
    s = z * np.exp(z) / (1 + np.exp(z))
    want = s * u
    d = np.abs(s) * du + 2.0 ** -23 * (6 + 1.173 * abs(z)) * np.abs(want) + abs(z) * np.abs(u) * 2.0 ** -126
    tol = d + 2.0 ** -8 * (np.abs(want) + d) + 2.0 ** -134
    assert np.all(np.abs(to_np(a).astype(np.float64) - want) <= tol)
