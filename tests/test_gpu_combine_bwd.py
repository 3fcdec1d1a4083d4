"""GPU parity of moe_unpermute_combine_bwd against the float64 oracle: dy_perm is
one product and its rounding; a dot product of h values passes at most h / 128 + 16
additions one after the other (U = 2^-24 of the sum of magnitudes each)."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu, to_dev, to_np
from oracle import fp8_oracle as X

pytestmark = [pytest.mark.gpu, needs_gpu]

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def _case(T, h, E, K, dtype, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :K]
    flat = np.argsort(idx.ravel(), kind="stable")
    keep = rng.random(T * K) >= drop
    dst = np.full(T * K, -1, np.int32)
    kept = [p for p in flat if keep[p]]
    dst[kept] = np.arange(len(kept))
    w = rng.random((T, K)).astype(np.float32)
    dt = lambda a: to_np(to_dev(a, dtype))  # noqa: E731
    return dst.reshape(T, K), w, dt(rng.standard_normal((T, h))), dt(rng.standard_normal((T * K, h)))


def _check(M, dst, w, dy, yp, dtype):
    T, K = dst.shape
    h = dy.shape[1]
    cfg = M.make_config(T, h, max(K, 1), K, 8, dtype=M.MOE_BF16 if dtype == "bf16" else M.MOE_F32)
    out = to_dev(np.full((T * K, h), 33.0), dtype)
    dw = torch.full((T, K), 77.0, device="cuda")
    dd, dyd, ypd = torch.from_numpy(dst).cuda(), to_dev(dy, dtype), to_dev(yp, dtype)
    wd = None if w is None else to_dev(w, "f32")
    M.moe_unpermute_combine_bwd(cfg, dyd, ypd, dd, wd, out, dw)
    assert M.moe_get_error() == M.MOE_OK
    ww = np.ones((T, K)) if w is None else w
    rp, rw = X.combine_bwd(dy, yp, dst, ww, np.full((T * K, h), 33.0))
    assert np.all(np.abs(to_np(out) - rp) <= (HALF[dtype] + 2 * U) * np.abs(rp))
    S = np.abs(np.where(dst >= 0, (np.abs(dy)[:, None, :] * np.abs(yp)[np.maximum(dst, 0)]).sum(2), 0.0))
    assert np.all(np.abs(to_np(dw) - rw) <= (h / 128 + 16) * U * S)
    assert torch.all(dw[torch.from_numpy(dst).cuda() < 0] == 0)
    alone = to_dev(np.full((T * K, h), 33.0), dtype)
    M.moe_unpermute_combine_bwd(cfg, dyd, None, dd, wd, alone)          # rows alone: the same bits
    assert torch.equal(alone, out)
    dw2 = torch.empty_like(dw)
    M.moe_unpermute_combine_bwd(cfg, dyd, ypd, dd, wd, alone, dw2)
    assert torch.equal(dw, dw2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,h,E,K,drop", [(1, 8, 1, 1, 0.0), (1, 7168, 8, 8, 0.0), (333, 2048, 64, 8, 0.0),
                                          (77, 1000, 16, 16, 0.2), (300, 264, 5, 3, 0.5), (64, 4096, 2, 2, 0.0),
                                          (40, 128, 8, 6, 1.0), (9, 12000, 4, 4, 0.1)])
def test_matches_oracle(T, h, E, K, drop, dtype):
    M = lib()
    dst, w, dy, yp = _case(T, h, E, K, dtype, T + h + K, drop)
    _check(M, dst, w, dy, yp, dtype)
    if K <= 3:
        _check(M, dst, None, dy, yp, dtype)


def test_is_the_combines_gradient():
    """moe_unpermute_combine at w + t e, w - t e (linear in w): differences give dprob; and
    <dy, y> = <dy_perm, y_perm> for the rows."""
    M = lib()
    dst, w, dy, yp = _case(50, 256, 8, 4, "f32", 5)
    cfg = M.make_config(50, 256, 8, 4, 8, dtype=M.MOE_F32)
    dd, dyd, ypd = torch.from_numpy(dst).cuda(), to_dev(dy, "f32"), to_dev(yp, "f32")
    y = torch.empty(50, 256, device="cuda")
    out, dw = torch.empty(200, 256, device="cuda"), torch.empty(50, 4, device="cuda")
    M.moe_unpermute_combine_bwd(cfg, dyd, ypd, dd, to_dev(w, "f32"), out, dw)

    def loss(w_):
        M.moe_unpermute_combine(cfg, ypd, dd, to_dev(w_, "f32"), None, y)
        return float((to_np(y).astype(np.float64) * dy).sum())

    S = float((np.abs(w)[:, :, None] * np.abs(yp[dst]) * np.abs(dy)[:, None, :]).sum())
    assert abs(loss(w) - float((to_np(out).astype(np.float64) * yp).sum())) <= 8 * U * S
    e = np.random.default_rng(6).standard_normal(w.shape).astype(np.float32)
    got = (loss(w + 0.5 * e) - loss(w - 0.5 * e))
    tol = 8 * U * (S + float((np.abs(e)[:, :, None] * np.abs(yp[dst]) * np.abs(dy)[:, None, :]).sum()))
    assert abs(got - float((to_np(dw).astype(np.float64) * e).sum())) <= 4 * tol


def test_dispatch_gradient_is_the_combine_without_weights():
    """dx[t] = sum_k dx_perm[dst_row[t, k]]: the gradient of moe_permute's copies."""
    M = lib()
    dst, _, _, dxp = _case(60, 512, 16, 6, "bf16", 7, drop=0.1)
    cfg = M.make_config(60, 512, 16, 6, 8)
    dx = torch.empty(60, 512, dtype=torch.bfloat16, device="cuda")
    M.moe_unpermute_combine(cfg, to_dev(dxp, "bf16"), torch.from_numpy(dst).cuda(), None, None, dx)
    want = X.combine(dxp, dst, np.ones(dst.shape))
    S = X.combine(np.abs(dxp), dst, np.ones(dst.shape))
    assert np.all(np.abs(to_np(dx) - want) <= 2.0 ** -8 * np.abs(want) + 8 * U * S)


def test_bad_rows_are_reported_and_skipped():
    M = lib()
    dst, w, dy, yp = _case(20, 64, 4, 2, "bf16", 8)
    bad = dst.copy()
    bad[3, 1], bad[7, 0] = 40, -5                     # P = 40 rows
    cfg = M.make_config(20, 64, 4, 2, 8)
    out = torch.full((40, 64), 33.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((20, 2), 77.0, device="cuda")
    M.moe_unpermute_combine_bwd(cfg, to_dev(dy, "bf16"), to_dev(yp, "bf16"), torch.from_numpy(bad).cuda(),
                                to_dev(w, "f32"), out, dw)
    assert M.moe_get_error() == M.MOE_ERR_DEVICE_BOUNDS and M.moe_get_error() == M.MOE_OK
    assert dw[3, 1] == 0 and dw[7, 0] == 0
    assert torch.all(out[int(dst[3, 1])] == 33.0) and torch.all(out[int(dst[7, 0])] == 33.0)
    assert torch.isfinite(dw).all() and (dw == 77.0).sum() == 0


def test_no_tokens():
    M = lib()
    M.moe_unpermute_combine_bwd(M.make_config(0, 64, 4, 2, 8), None, None, None, None, None)
    assert M.moe_get_error() == M.MOE_OK
