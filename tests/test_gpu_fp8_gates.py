"""moe_expert_fc1_fp8 with strongly negative gates, where SiLU decays to nothing.

Tokens of ones and gate weights of one value make a gate z the same exact number in
every product order.  CUDA bounds expf by 2 units in the last place and __fdividef by
2 (a unit is 2^-23 of the value); the sum, the two products and p round once each:
2^-23 (4 + 2) of a in all.  A quotient below 2^-126 may come out as 0: another
|z u| 2^-126.  The bf16 output adds half a step: 2^-8 of the value, or half of the
smallest subnormal, 2^-134."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu, to_np
from oracle import fp8_oracle as X
from test_gpu_fp8 import U, bf16, quantize_dev, weights_dev

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("P", [5, 300])
@pytest.mark.parametrize("z", [-8.0, -24.0, -48.0, -64.0, -96.0, -128.0, -768.0])
def test_strongly_negative_gates(z, P):
    M = lib()
    h, F = 128, 256
    rng = np.random.default_rng(int(-z))
    w1 = np.empty((2 * F, h), np.float32)
    w1[:F] = z / h                                   # a power of two times 1, 1.5: exact
    w1[F:] = bf16(rng.standard_normal((F, h)))
    cfg = M.make_config(P, h, 1, 1, F)
    od = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    xq, xsf = quantize_dev(M, np.ones((P, h), np.float32))
    wq, wsf = weights_dev(M, w1, 1)
    a = torch.full((P, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    M.moe_expert_fc1_fp8(cfg, xq, xsf, od, None, wq, wsf, None, a, None, None)
    assert M.moe_get_error() == M.MOE_OK
    # 1 / 448 and |z| / (448 h) are fp32 scales of the codes 448: their product with 448^2 is
    # within 3 half steps of z
    x = X.dequantize(*X.quantize(np.ones((1, h))))
    w = X.dequantize(*X.quantize(w1, True))
    g = (x @ w[:F].T)[0]
    assert np.all(np.abs(g - z) <= 2.0 ** -22 * abs(z))
    u = (x @ w[F:].T)[0]
    du = (128 + 6) * U * (np.abs(x) @ np.abs(w[F:]).T)[0]
    dg = (128 + 6) * U * abs(z)                      # moves exp(z) by that share
    s = g * np.exp(g) / (1 + np.exp(g))
    want = s * u
    d = np.abs(s) * du + (np.expm1(dg) * 1.1 + 6 * U) * (np.abs(want) + np.abs(s) * du) + abs(z) * (np.abs(u) + du) * 2.0 ** -126
    tol = d + 2.0 ** -8 * (np.abs(want) + d) + 2.0 ** -134
    assert np.all(np.abs(to_np(a).astype(np.float64) - want) <= tol)
