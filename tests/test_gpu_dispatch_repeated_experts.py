"""Dispatch maps of large tables in which tokens name an expert twice: the maps by the rule
(a pair's row is its expert's offset plus the pairs of earlier tokens), on both paths of the
scan, and their time beside a table without such tokens (1.1 times as long; with 9 ballots
for each pair of a token's slots it was 2.3 times)."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]


def _table(T, E, K, seed, repeats):
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)
    if repeats:  # one token or more in every 32
        idx[::17, K - 1] = idx[::17, 0]
        idx[5::32, :] = idx[5::32, :1]
    return idx


class Maps:
    def __init__(self, M, idx, E, cap=0):
        T, K = idx.shape
        i32 = dict(dtype=torch.int32, device="cuda")
        self.M, self.idx = M, torch.from_numpy(idx).cuda()
        self.cfg = M.make_config(T, 128, E, K, 128, capacity=cap)
        self.ws = torch.empty(M.moe_workspace_size(self.cfg), dtype=torch.uint8, device="cuda")
        self.counts, self.offsets, self.dst = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T, K, **i32)
        self.src = torch.full((T * K,), -7, **i32)
        self.prob, self.perm_prob = torch.rand(T, K, device="cuda"), torch.full((T * K,), -1.0, device="cuda")

    def run(self):
        self.M.moe_permute(self.cfg, None, self.idx, self.prob, None, self.counts, self.offsets, self.dst, self.src,
                           self.perm_prob, self.ws)


@pytest.mark.parametrize("T,E,K,cap", [(5000, 256, 8, 0), (1000, 8, 4, 0), (40000, 64, 16, 0), (6000, 128, 6, 100),
                                       (33, 256, 16, 0), (9000, 3, 2, 0)])
def test_maps(T, E, K, cap):
    M = lib()
    idx = _table(T, E, max(1, K), T, True) if K <= E else None
    m = Maps(M, idx, E, cap)
    m.run()
    assert M.moe_get_error() == M.MOE_OK
    count = np.zeros((T + 1, E), np.int64)
    np.add.at(count, (np.repeat(np.arange(T), K) + 1, idx.ravel()), 1)
    before = np.cumsum(count, axis=0)[:-1]                      # pairs of earlier tokens, [T, E]
    pos = np.take_along_axis(before, idx.astype(np.int64), axis=1)
    kept = np.minimum(before[-1] + count[-1], cap or T * K)
    off = np.concatenate([[0], np.cumsum(kept)])
    dst = np.where((pos < cap) if cap else True, off[idx] + pos, -1)
    np.testing.assert_array_equal(m.counts.cpu().numpy(), kept)
    np.testing.assert_array_equal(m.offsets.cpu().numpy(), off)
    np.testing.assert_array_equal(m.dst.cpu().numpy(), dst)
    src = np.full(T * K, -7)
    ok = dst >= 0
    src[dst[ok]] = np.repeat(np.arange(T), K).reshape(T, K)[ok]
    np.testing.assert_array_equal(m.src.cpu().numpy(), src)
    pp, prob = np.full(T * K, -1.0, np.float32), m.prob.cpu().numpy()
    for k in range(K):                                          # of a row's slots the last one's
        pp[dst[ok[:, k], k]] = prob[ok[:, k], k]
    np.testing.assert_array_equal(m.perm_prob.cpu().numpy(), pp)


def test_time_beside_a_table_without_repeats():
    M = lib()
    T, E, K = 16384, 256, 16
    maps = [Maps(M, _table(T, E, K, 1, r), E) for r in (False, True)]
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))

    def us(m):
        begin.record()
        for _ in range(20):
            m.run()
        end.record()
        end.synchronize()
        return begin.elapsed_time(end) * 50

    for m in maps:
        us(m)
    plain, repeated = (sorted(t)[5] for t in zip(*[[us(m) for m in maps] for _ in range(11)]))
    print(f"{plain:.1f} us, with repeats {repeated:.1f}")
    assert repeated < 2 * plain, (plain, repeated)
