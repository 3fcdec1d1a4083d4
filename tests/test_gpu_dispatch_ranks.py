"""Dispatch maps of index tables that no router of the library makes but a caller may:
tokens that name an expert twice, ids outside the experts, one expert for all.  A pair's
row is its expert's offset plus the number of pairs of earlier tokens with that expert (so
the two pairs of a token that names one twice share a row, and the next row stays free)."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]


def _maps(idx, E, cap):
    T, K = idx.shape
    ok = (idx >= 0) & (idx < E)
    counts = np.bincount(idx[ok], minlength=E)
    kept = np.minimum(counts, cap) if cap else counts
    off = np.concatenate([[0], np.cumsum(kept)])
    seen, dst = np.zeros(E, np.int64), np.full((T, K), -1)
    for t in range(T):
        for k in range(K):
            e = idx[t, k]
            if ok[t, k] and not (cap and seen[e] >= cap):
                dst[t, k] = off[e] + seen[e]
        np.add.at(seen, idx[t][ok[t]], 1)
    return kept, off, dst


@pytest.mark.parametrize("T,E,K,cap,kind", [(70, 8, 4, 0, "twice"), (3000, 256, 8, 0, "twice"), (100, 256, 8, 0, "free"),
                                            (4000, 64, 6, 0, "free"), (500, 8, 4, 60, "twice"), (333, 5, 2, 0, "outside"),
                                            (33, 3, 2, 0, "one"), (1, 256, 16, 0, "free"), (900, 16, 16, 0, "free")])
def test_maps(T, E, K, cap, kind):
    M = lib()
    rng = np.random.default_rng(T + E)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :K]
    if kind == "twice":
        rows = rng.choice(T, max(1, T // 10), replace=False)
        idx[rows, 1] = idx[rows, 0]
        idx[rows[0]] = idx[rows[0], 0]
    elif kind == "outside":
        idx[5, 0], idx[T - 1, 1] = -1, E
    elif kind == "one":
        idx[:, 0], idx[:, 1] = 2, 0
    idx = idx.astype(np.int32)
    counts, off, dst = _maps(idx, E, cap)
    cfg = M.make_config(T, 128, E, K, 128, capacity=cap)
    ws = torch.empty(M.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    c, o, d = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T, K, **i32)
    s, p = torch.full((T * K,), -7, **i32), torch.full((T * K,), -1.0, device="cuda")
    prob = torch.rand(T, K, device="cuda")
    M.moe_permute(cfg, None, torch.from_numpy(idx).cuda(), prob, None, c, o, d, s, p, ws)
    assert M.moe_get_error() == (M.MOE_ERR_DEVICE_BOUNDS if kind == "outside" else M.MOE_OK)
    np.testing.assert_array_equal(c.cpu().numpy(), counts)
    np.testing.assert_array_equal(o.cpu().numpy(), off)
    np.testing.assert_array_equal(d.cpu().numpy(), dst)
    src, pp, ph = s.cpu().numpy(), p.cpu().numpy(), prob.cpu().numpy()
    for t, k in zip(*np.nonzero(dst >= 0)):
        assert src[dst[t, k]] == t and pp[dst[t, k]] in ph[t]
    free = np.setdiff1d(np.arange(T * K), dst[dst >= 0])
    assert np.all(src[free] == -7) and np.all(pp[free] == -1.0)
