"""The combine's gradient where slots of one token share a row, which moe_permute's maps
have for a token that names an expert twice: the combine adds such a row once for each
slot, so its gradient is the sum of their weights times dy.

Tolerance: the sum of at most K weights is off by at most K U of itself (they are positive,
U = 2^-24), the product by U, the output's rounding by half a step of its type.  A dot
product adds the values of ceil(h / (32 V W)) vectors of V in a thread, 5 times in a warp and
once for each of the token's W warps (1 below 128 vectors a row, 2 below 256, else 4 or, for
at most two tokens an SM, 16)."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu, to_dev, to_np

pytestmark = [pytest.mark.gpu, needs_gpu]

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def _maps(M, T, E, K, seed):
    """moe_permute's rows for a table in which every third token names an expert several times."""
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)
    idx[::3, K - 1] = idx[::3, 0]
    idx[::9] = idx[::9, :1]
    cfg = M.make_config(T, 128, E, K, 128)
    ws = torch.empty(M.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    dst = torch.empty(T, K, **i32)
    M.moe_permute(cfg, None, torch.from_numpy(idx).cuda(), None, None, torch.empty(E, **i32), torch.empty(E + 1, **i32),
                  dst, torch.empty(T * K, **i32), None, ws)
    torch.cuda.synchronize()
    return dst


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,h,E,K", [(1, 8, 4, 2), (40, 264, 8, 2), (33, 1000, 5, 3), (400, 2048, 64, 8), (50, 7168, 16, 16),
                                     (700, 4096, 8, 4)])
def test_weights_of_shared_rows_add_up(T, h, E, K, dtype):
    M = lib()
    dst = _maps(M, T, E, K, T + h)
    dh = dst.cpu().numpy()
    rng = np.random.default_rng(h)
    cfg = M.make_config(T, h, E, K, 8, dtype=M.MOE_BF16 if dtype == "bf16" else M.MOE_F32)
    dy, yp = (to_dev(rng.standard_normal(s), dtype) for s in ((T, h), (T * K, h)))
    w = rng.uniform(0.05, 1.0, (T, K)).astype(np.float32)
    for weights in (w, None):
        out = to_dev(np.full((T * K, h), 33.0), dtype)
        dw = torch.full((T, K), 77.0, device="cuda")
        M.moe_unpermute_combine_bwd(cfg, dy, yp, dst, None if weights is None else to_dev(w, "f32"), out, dw)
        assert M.moe_get_error() == M.MOE_OK
        total = np.zeros((T * K, 1))
        rows = np.zeros((T * K, h))
        np.add.at(total, (dh.ravel(), 0), (np.ones_like(w) if weights is None else w).astype(np.float64).ravel())
        rows[dh.ravel()] = np.repeat(to_np(dy).astype(np.float64), K, axis=0)
        named = np.zeros(T * K, bool)
        named[dh.ravel()] = True
        want, got = (total * rows)[named], to_np(out)
        assert np.all(np.abs(got[named] - want) <= (HALF[dtype] + (K + 2) * U) * np.abs(want))
        assert np.all(got[~named] == 33.0)
        # the combine's own pairing, <dy, y> = <dy_perm, y_perm>, over the rows that it reads
        y = torch.empty_like(dy)
        M.moe_unpermute_combine(cfg, yp, dst, None if weights is None else to_dev(w, "f32"), None, y)
        left = (to_np(dy).astype(np.float64) * to_np(y)).sum()
        right = (got[named].astype(np.float64) * to_np(yp)[named]).sum()
        S = (np.abs(want) * np.abs(to_np(yp)[named])).sum()
        assert abs(left - right) <= 2 * (HALF[dtype] + (2 * K + 2) * U) * S
        # each slot's dot product is with its row, shared or not
        V = 8 if dtype == "bf16" else 4
        vecs, sms = h // V, torch.cuda.get_device_properties(0).multi_processor_count
        W = 1 if vecs < 128 else 2 if vecs < 256 else 4 if T > 2 * sms else 16
        adds = V * -(-vecs // (32 * W)) + 5 + W
        dots = (to_np(dy).astype(np.float64)[:, None, :] * to_np(yp)[dh]).sum(2)
        mags = (np.abs(to_np(dy))[:, None, :] * np.abs(to_np(yp))[dh]).sum(2)
        assert np.all(np.abs(to_np(dw) - dots) <= adds * U * mags)
