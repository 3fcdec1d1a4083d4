"""The FP8 products with several tiles a thread block, where accumulators, scale groups,
barriers' phases and the 8-bit outputs' meetings carry over from one tile to the next: odd
numbers of 128-column blocks, ones that leave a group of eight scales unfilled, an odd
number of FC2's column blocks; ragged and empty experts.  Rows of every expert against the
values that the codes stand for, in 64 bits, with test_gpu_fp8's tolerances; then every row
of every output against calls of so few rows that no block has a second tile, bit for bit."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu
from oracle import fp8_oracle as X
from oracle.mxfp8_oracle import e4m3_decode
from test_gpu_fp8 import U, _fc1_bound, _near, f32, u8

pytestmark = [pytest.mark.gpu, needs_gpu]


def _rows_of_interest(rng, offs, n=160):
    """Every expert's first and last row and its tiles' edges, and others at random."""
    rows = [rng.integers(offs[0], offs[-1], n)]
    for lo, hi in zip(offs[:-1], offs[1:]):
        if hi > lo:
            rows.append([lo, hi - 1, min(lo + 127, hi - 1), min(lo + 128, hi - 1), lo + (hi - lo - 1) // 128 * 128])
    return np.unique(np.concatenate(rows))


def _z(A, offs, q, sf):
    """The products in 64 bits of rows sorted by expert and how far the GPU's may be from them."""
    E, N, K = q.shape
    z, t = np.zeros((A.shape[0], N)), np.zeros((A.shape[0], N))
    for e in range(E):
        r = slice(int(offs[e]), int(offs[e + 1]))
        if r.stop > r.start:
            W = X.dequantize(q[e].cpu().numpy(), sf[e].cpu().numpy())
            z[r] = A[r] @ W.T
            t[r] = (128 + K / 128 + 4) * U * (np.abs(A[r]) @ np.abs(W).T)
    return z, t


class Products:
    def __init__(self, M, P, E, h, F, empty):
        self.M, self.P, self.E, self.h, self.F = M, P, E, h, F
        self.rng = rng = np.random.default_rng(P + h)
        share = rng.dirichlet(np.full(E, 2.0))
        share[list(empty)] = 0.0
        self.offs = np.concatenate([[0], np.cumsum(rng.multinomial(P, share / share.sum()))]).astype(np.int64)
        self.few = P <= 16 * E
        g = torch.Generator(device="cuda").manual_seed(P + F)
        n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        x = (n(P, h) * torch.exp2(torch.randint(-6, 6, (P, 1), device="cuda", generator=g))).bfloat16()
        self.xq, self.xsf = u8(P, h), f32(P, h // 128)
        M.moe_fp8_quantize(P, h, x, self.xq, self.xsf)
        self.w = []
        for N, K in ((2 * F, h), (h, F)):
            q, sf = u8(E, N, K), f32(E, N // 128, K // 128)
            M.moe_fp8_quantize_weights(E, N, K, (n(E, N, K) / K ** 0.5).bfloat16(), q, sf)
            self.w += [q, sf]
        self.p = 0.05 + 0.95 * torch.rand(P, device="cuda", generator=g)

    def tiles(self):
        """Of FC1 and FC2."""
        r = int((-(-np.diff(self.offs) // (16 if self.few else 128))).sum())
        return r * (self.F // 128), r * (self.h // 128 if self.few else -(-self.h // 256))

    def run(self, xq, xsf, p, offs, w):
        n, E = xq.shape[0], len(offs) - 1
        cfg = self.M.make_config(n, self.h, E, 1, self.F)
        od = torch.tensor(offs, dtype=torch.int32, device="cuda")
        full = lambda k: torch.full((n, k), 33.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        o = dict(save=full(2 * self.F), a=full(self.F), aq=u8(n, self.F), asf=f32(n, self.F // 128), y=full(self.h))
        self.M.moe_expert_fc1_fp8(cfg, xq, xsf, od, p, w[0], w[1], o["save"], o["a"], o["aq"], o["asf"])
        self.M.moe_expert_fc2_fp8(cfg, o["aq"], o["asf"], od, w[2], w[3], o["y"])
        return o

    def check(self, o):
        s = _rows_of_interest(self.rng, self.offs)
        so, g = np.searchsorted(s, self.offs), torch.from_numpy(s).cuda()
        np_ = lambda t: t[g].cpu().numpy()  # noqa: E731
        H, t = _z(X.dequantize(np_(self.xq), np_(self.xsf)), so, self.w[0], self.w[1])
        a, d = _fc1_bound(H, t, np_(self.p))
        _near(o["save"][g], H, t + 2.0 ** -8 * (np.abs(H) + t) + 1e-30)
        _near(o["a"][g], a, d + 2.0 ** -8 * (np.abs(a) + d))
        sf = np_(o["asf"]).astype(np.float64)
        sc = np.repeat(sf, 128, 1)
        deq = e4m3_decode(np_(o["aq"])) * sc
        assert np.all(np.abs(deq - a) <= d + np.maximum(2.0 ** -4 * (np.abs(a) + d), 2.0 ** -10 * sc) * (1 + 2.0 ** -20))
        top, dtop = (v.reshape(len(s), -1, 128).max(2) for v in (np.abs(a), d))
        assert np.all(np.abs(sf * 448 - top) <= dtop + 2.0 ** -22 * top)
        y, ty = _z(deq, so, self.w[2], self.w[3])
        _near(o["y"][g], y, ty + 2.0 ** -8 * (np.abs(y) + ty) + 1e-30)

    def check_tile_by_tile(self, o, sms):
        unit, E = (16, self.E) if self.few else (128, 1)
        step = unit * (sms // max(self.F // 128, self.h // 128 if self.few else -(-self.h // 256)))
        assert step > 0
        for e in range(self.E):
            # the same kernel: all experts in name where it is the one for few rows an expert
            w = self.w if self.few else [t[e].clone() for t in self.w]
            for lo in range(int(self.offs[e]), int(self.offs[e + 1]), step):
                r = slice(lo, min(lo + step, int(self.offs[e + 1])))
                n = r.stop - lo
                if not self.few and n <= 16:
                    continue                                            # (so few would take the other one)
                at = [0] * (e + 1 if self.few else 1)
                alone = self.run(self.xq[r], self.xsf[r].clone(), self.p[r], at + [n] * (E + 1 - len(at)), w)
                for name, v in alone.items():
                    assert torch.equal(v, o[name][r]), (name, e, lo)


@pytest.mark.parametrize("P,E,h,F,empty,few", [
    (9000, 8, 1664, 1920, (), False),          # 13 and 15 blocks of K
    (20000, 16, 640, 896, (0, 9), False),      # 5 and 7
    (60000, 3, 128, 512, (), False),           # one and four, an odd last column tile of FC2 alone
    (1024, 64, 384, 640, (3, 60), True),       # units of 16 rows: 3 and 5
    (512, 32, 1152, 1664, (), True),           # 9 and 13
])
def test_products(P, E, h, F, empty, few):
    M = lib()
    c = Products(M, P, E, h, F, empty)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert c.few == few and c.tiles()[0] >= 3 * sms - 8 and c.tiles()[1] > 1.5 * sms, c.tiles()
    o = c.run(c.xq, c.xsf, c.p, c.offs.tolist(), c.w)
    assert M.moe_get_error() == M.MOE_OK
    c.check(o)
    c.check_tile_by_tile(o, sms)
    again = c.run(c.xq, c.xsf, c.p, c.offs.tolist(), c.w)
    for name, v in again.items():
        assert torch.equal(v, o[name]), name
    assert M.moe_get_error() == M.MOE_OK
