"""GPU parity of FP8 with a scale for each block of 128: the quantisers bit-exact
against the oracle, the dispatch of 8-bit rows, the grouped products, and the whole
path as it is used.

Tolerances of the products: the operands' values are exact.  A block of 128
products is summed on the tensor cores, at most one unit of the last place (U =
2^-23) of the sum of magnitudes an addition; a block's sum then meets its scales
(rounded to fp32) and K / 128 such sums are added in fp32: |gpu - exact| <=
(128 + K / 128 + 4) U sum_k |a_k w_k|, and a bf16 output adds half a step, 2^-8
of it.  FC1 carries the bound of gate and up through p silu(g) u with |silu'| <=
1.1, plus 2^-18 |a| for the fp32 evaluation."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu, to_dev, to_np
from oracle import fp8_oracle as X
from oracle.mxfp8_oracle import e4m3_decode, silu

pytestmark = [pytest.mark.gpu, needs_gpu]

U = 2.0 ** -23


def bf16(a):
    return to_np(torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16))


def u8(*s, fill=0xEE):
    return torch.full(s, fill, dtype=torch.uint8, device="cuda")


def f32(*s, fill=77.0):
    return torch.full(s, fill, device="cuda")


def quantize_dev(M, x):
    q, sf = u8(*x.shape), f32(x.shape[0], x.shape[1] // 128)
    M.moe_fp8_quantize(x.shape[0], x.shape[1], to_dev(x, "bf16"), q, sf)
    return q, sf


def weights_dev(M, w, E):
    N, K = w.shape[0] // E, w.shape[1]
    q, sf = u8(E, N, K), f32(E, N // 128, K // 128)
    M.moe_fp8_quantize_weights(E, N, K, to_dev(w, "bf16"), q, sf)
    return q, sf


def hard_rows(rng, rows, K):
    """A wide range, zero blocks, subnormals, exact ties, the largest values, non-finite ones."""
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-60, 60, (rows, 1)))
    if rows > 8:
        x[1, :128] = 0.0
        x[2, :128] = rng.standard_normal(128) * 2.0 ** -130
        grid = e4m3_decode(np.arange(127))
        x[3, :128] = np.concatenate([[448.0], rng.choice((grid[1:] + grid[:-1]) / 2, 127)]) * 2.0 ** 5
        x[4, 5], x[5, K - 1], x[6, 3] = np.inf, np.nan, -np.inf
        x[7, :128] = rng.standard_normal(128) * 1e38
        x[7, 0] = 3.38e38
        x[8, :128] = rng.standard_normal(128) * 2.0 ** -118
    return bf16(x)


@pytest.mark.parametrize("rows,K", [(1, 128), (300, 256), (1021, 2048), (37, 7168), (9, 14336), (2000, 384)])
def test_quantize_bit_exact(rows, K):
    M = lib()
    x = hard_rows(np.random.default_rng(rows), rows, K)
    q, sf = quantize_dev(M, x)
    oq, osf = X.quantize(x)
    np.testing.assert_array_equal(sf.cpu().numpy(), osf)
    np.testing.assert_array_equal(q.cpu().numpy(), oq)


def test_quantize_every_ratio_of_mantissas():
    """Every 8-bit mantissa beside every 8-bit largest one, at code exponents from the
    subnormals to the top: what lies on the border of two codes goes to the even one."""
    M = lib()
    m = np.arange(128, 256, dtype=np.float64)
    x = np.zeros((128 * 20, 128))
    for e in range(20):
        x[e * 128:(e + 1) * 128, :] = m[None, :] * 2.0 ** -e
        x[e * 128:(e + 1) * 128, 0] = m if e else 2 * m
    x = bf16(x)
    q, sf = quantize_dev(M, x)
    oq, osf = X.quantize(x)
    np.testing.assert_array_equal(q.cpu().numpy(), oq)
    np.testing.assert_array_equal(sf.cpu().numpy(), osf)


@pytest.mark.parametrize("G,N,K", [(1, 128, 128), (3, 256, 384), (8, 128, 2048), (2, 1024, 640), (64, 128, 128)])
def test_quantize_weights_bit_exact(G, N, K):
    M = lib()
    rng = np.random.default_rng(G * N + K)
    w = rng.standard_normal((G * N, K)) * np.exp2(rng.integers(-8, 8, (G * N, 1)))
    w[0, 0] = 0.0
    if G > 1:
        w[N:N + 128, :128] = 0.0
        w[2 * N - 1, K - 1] = np.inf
    w = bf16(w)
    q, sf, qt, sft = u8(G, N, K), f32(G, N // 128, K // 128), u8(G, K, N), f32(G, K // 128, N // 128)
    M.moe_fp8_quantize_weights(G, N, K, to_dev(w, "bf16"), q, sf, qt, sft)
    oq, osf = X.quantize(w, tall=True)
    oq, osf = oq.reshape(G, N, K), osf.reshape(G, N // 128, K // 128)
    np.testing.assert_array_equal(sf.cpu().numpy(), osf)
    np.testing.assert_array_equal(q.cpu().numpy(), oq)
    np.testing.assert_array_equal(sft.cpu().numpy(), osf.transpose(0, 2, 1))
    np.testing.assert_array_equal(qt.cpu().numpy(), oq.transpose(0, 2, 1))
    q2, sf2 = weights_dev(M, w, G)
    assert torch.equal(q2, q) and torch.equal(sf2.view(torch.int32), sf.view(torch.int32))


# ---- dispatch ------------------------------------------------------------------------
def _maps(M, T, E, K):
    i = dict(dtype=torch.int32, device="cuda")
    return dict(counts=torch.empty(E, **i), offsets=torch.empty(E + 1, **i), dst_row=torch.empty(T, K, **i),
                src_token=torch.full((T * K,), -9, **i), perm_prob=f32(T * K))


@pytest.mark.parametrize("T,h,E,K,capacity", [(1, 128, 1, 1, 0), (333, 2048, 64, 8, 0), (1000, 384, 8, 2, 0),
                                              (257, 7168, 16, 3, 0), (50, 1152, 256, 16, 0), (400, 256, 8, 4, 150)])
def test_permute_fp8(T, h, E, K, capacity):
    """The maps of moe_permute, and its rows if the dequantised codes were permuted."""
    M = lib()
    rng = np.random.default_rng(T + h)
    idx = torch.from_numpy(np.argsort(rng.random((T, E)) * np.arange(1, E + 1), axis=1)[:, :K].astype(np.int32)).cuda()
    prob = torch.rand(T, K, device="cuda")
    xq = torch.from_numpy(rng.integers(0, 256, (T, h), dtype=np.uint8)).cuda()
    xsf = torch.rand(T, h // 128, device="cuda")
    cfg = M.make_config(T, h, E, K, 128, capacity=capacity)
    ws = torch.empty(M.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    a, b = _maps(M, T, E, K), _maps(M, T, E, K)
    x = torch.zeros(T, h, dtype=torch.bfloat16, device="cuda")
    xp = torch.empty(T * K, h, dtype=torch.bfloat16, device="cuda")
    M.moe_permute(cfg, x, idx, prob, xp, ws=ws, **a)
    q, sf = u8(T * K, h), f32(T * K, h // 128)
    M.moe_permute_fp8(cfg, xq, xsf, idx, prob, q, sf, ws=ws, **b)
    assert M.moe_get_error() == M.MOE_OK
    n = int(a["offsets"][-1])
    assert (n < T * K) == (capacity > 0)
    for k in a:
        rows = slice(0, n) if k in ("src_token", "perm_prob") else slice(None)
        assert torch.equal(a[k][rows], b[k][rows]), k
    src = b["src_token"][:n].long()
    assert torch.equal(q[:n], xq[src]) and torch.equal(sf[:n], xsf[src])
    assert torch.all(q[n:] == 0xEE) and torch.all(sf[n:] == 77.0)      # rows of no slot


# ---- products ---------------------------------------------------------------------------
def _case(seed, T, K, E, h, F, skew=False, empty=()):
    rng = np.random.default_rng(seed)
    P = T * K
    w = rng.dirichlet(np.full(E, 0.3)) if skew else np.ones(E)
    for e in empty:
        w[e] = 0.0
    offsets = np.concatenate([[0], np.cumsum(rng.multinomial(P, w / w.sum()))]).astype(np.int64)
    rows = np.exp2(rng.integers(-6, 6, (P, 1)))           # rows and blocks of differing scales
    return dict(T=T, K=K, E=E, h=h, F=F, P=P, offsets=offsets, x=bf16(rng.standard_normal((P, h)) * rows),
                w1=bf16(rng.standard_normal((E * 2 * F, h)) / np.sqrt(h) *
                        np.repeat(np.exp2(rng.integers(-3, 3, (1, h // 128))), 128, 1)),
                w2=bf16(rng.standard_normal((E * h, F)) / np.sqrt(F)),
                p=rng.uniform(0.05, 1.0, P).astype(np.float32))


def _z(A, offs, W, Nw, Kd):
    return (X.grouped_product(A, offs, W, Nw),
            (128 + Kd / 128 + 4) * U * X.grouped_product(np.abs(A), offs, np.abs(W), Nw))


def _fc1_bound(H, t, p):
    F = H.shape[1] // 2
    g, u, tg, tu = H[:, :F], H[:, F:], t[:, :F], t[:, F:]
    pp = np.asarray(p, np.float64)[:, None]
    a = pp * silu(g) * u
    d = pp * (1.1 * tg * (np.abs(u) + tu) + (np.abs(silu(g)) + 1.1 * tg) * tu)
    return a, d + 2.0 ** -18 * np.abs(a) + 1e-30


def _near(got, want, tol):
    got = to_np(got).astype(np.float64)
    assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) / tol).max())


def _check_products(M, c, prob=True, used=None):
    """FC1 with every output, FC2 on the GPU's own 8-bit a; rows behind the last expert's untouched."""
    P, E, h, F, offs = c["P"], c["E"], c["h"], c["F"], c["offsets"]
    cfg = M.make_config(c["T"], h, E, c["K"], F)
    od = torch.from_numpy(offs.astype(np.int32)).cuda()
    n0, n1 = int(offs[0]), int(offs[-1])
    xq, xsf = quantize_dev(M, c["x"])
    w1q, w1sf = weights_dev(M, c["w1"], E)
    w2q, w2sf = weights_dev(M, c["w2"], E)
    full = lambda n: torch.full((P, n), 33.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    save, a, aq, asf, y = full(2 * F), full(F), u8(P, F), f32(P, F // 128), full(h)
    pd = torch.from_numpy(c["p"]).cuda() if prob else None
    M.moe_expert_fc1_fp8(cfg, xq, xsf, od, pd, w1q, w1sf, save, a, aq, asf)
    M.moe_expert_fc2_fp8(cfg, aq, asf, od, w2q, w2sf, y)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    A, W = X.dequantize(*X.quantize(c["x"])), X.dequantize(*X.quantize(c["w1"], True))
    H, t = _z(A, offs, W, 2 * F, h)
    a_ref, d = _fc1_bound(H, t, c["p"] if prob else np.ones(P))
    inside = slice(n0, n1)
    _near(save[inside], H[inside], (t + 2.0 ** -8 * (np.abs(H) + t) + 1e-30)[inside])
    _near(a[inside], a_ref[inside], (d + 2.0 ** -8 * (np.abs(a_ref) + d))[inside])
    s = asf.cpu().numpy().astype(np.float64)
    sc = np.repeat(s, 128, 1)
    deq = e4m3_decode(aq.cpu().numpy()) * sc
    tol = d + np.maximum(2.0 ** -4 * (np.abs(a_ref) + d), 2.0 ** -10 * sc) * (1 + 2.0 ** -20)
    assert np.all((np.abs(deq - a_ref) <= tol)[inside])
    top, dtop = (v.reshape(P, F // 128, 128).max(2) for v in (np.abs(a_ref), d))
    floor = 448 * 2.0 ** -125
    assert np.all((np.abs(s * 448 - np.maximum(top, floor)) <= dtop + 2.0 ** -22 * top)[inside])
    W2 = X.dequantize(*X.quantize(c["w2"], True))
    yr, ty = _z(np.where(np.isfinite(deq), deq, 0.0), offs, W2, h, F)
    _near(y[inside], yr[inside], (ty + 2.0 ** -8 * (np.abs(yr) + ty) + 1e-30)[inside])
    for t_, v in ((save, 33.0), (a, 33.0), (y, 33.0), (aq, 0xEE), (asf, 77.0)):
        assert torch.all(t_[:n0] == v) and torch.all(t_[n1:] == v)
    return save, a, aq, asf, y


CASES = [
    dict(seed=1, T=300, K=2, E=8, h=256, F=128),
    dict(seed=2, T=500, K=4, E=16, h=384, F=256, skew=True, empty=(3, 7)),
    dict(seed=3, T=100, K=8, E=64, h=512, F=128, skew=True),                 # experts below one tile
    dict(seed=4, T=2048, K=1, E=2, h=1024, F=384),                           # several tiles an expert
    dict(seed=5, T=1, K=1, E=3, h=128, F=128),                               # one row, one block
    dict(seed=6, T=1024, K=2, E=4, h=2048, F=640),
    dict(seed=7, T=1, K=8, E=256, h=1280, F=256),                            # one token
    dict(seed=8, T=13, K=8, E=64, h=2048, F=1024),
    dict(seed=9, T=64, K=2, E=8, h=1024, F=896),
    dict(seed=10, T=5, K=1, E=1, h=7168, F=128),                             # one expert
    dict(seed=11, T=40, K=6, E=8, h=640, F=128, skew=True),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: f"T{c['T']}_K{c['K']}_E{c['E']}_h{c['h']}_F{c['F']}")
def test_products_match_oracle(c):
    _check_products(lib(), _case(**c))


@pytest.mark.parametrize("n0,n1", [(0, 150), (17, 200), (60, 61), (100, 100)])
def test_rows_of_no_expert_are_left_alone(n0, n1):
    """Offsets that start behind row 0 and end before P (a padded batch, dropped slots)."""
    c = _case(21, 100, 2, 4, 256, 256)
    span = n1 - n0
    c["offsets"] = np.array([n0, n0 + span // 2, n0 + span // 2, n0 + span - span // 8, n1])
    _check_products(lib(), c)


def test_outputs_alone_null_prob_and_reruns_bitwise():
    M = lib()
    c = _case(22, 400, 2, 8, 256, 256, skew=True)
    save, a, aq, asf, _ = _check_products(M, c, prob=False)
    P, E, h, F = c["P"], c["E"], c["h"], c["F"]
    cfg = M.make_config(c["T"], h, E, c["K"], F)
    od = torch.from_numpy(c["offsets"].astype(np.int32)).cuda()
    xq, xsf = quantize_dev(M, c["x"])
    w1q, w1sf = weights_dev(M, c["w1"], E)
    for keep in (("a",), ("q",), ("save", "a"), ("save", "q"), ("a", "q")):
        s2 = torch.empty_like(save) if "save" in keep else None
        a2 = torch.empty_like(a) if "a" in keep else None
        q2, f2 = (torch.empty_like(aq), torch.empty_like(asf)) if "q" in keep else (None, None)
        M.moe_expert_fc1_fp8(cfg, xq, xsf, od, None, w1q, w1sf, s2, a2, q2, f2)
        for got, want in ((s2, save), (a2, a), (q2, aq), (f2, asf)):
            assert got is None or torch.equal(got, want), keep


@pytest.mark.parametrize("T,K", [(200, 1), (6, 2)])
def test_non_finite_rows_stay_in_their_rows(T, K):
    """A row with an infinity or a NaN is NaN in its own outputs and nowhere else."""
    M = lib()
    c = _case(23, T, K, 4, 256, 128)
    P, E, h, F = c["P"], c["E"], c["h"], c["F"]
    cfg = M.make_config(T, h, E, K, F)
    od = torch.from_numpy(c["offsets"].astype(np.int32)).cuda()
    w1q, w1sf = weights_dev(M, c["w1"], E)
    bad = [2, P - 2]
    outs = []
    for x in (c["x"], c["x"].copy()):
        if outs:
            x[bad[0], 3], x[bad[1], 200] = np.inf, np.nan
        xq, xsf = quantize_dev(M, x)
        a, q, sf = torch.zeros(P, F, dtype=torch.bfloat16, device="cuda"), u8(P, F), f32(P, F // 128)
        M.moe_expert_fc1_fp8(cfg, xq, xsf, od, None, w1q, w1sf, None, a, q, sf)
        outs.append((to_np(a), q.cpu().numpy(), sf.cpu().numpy()))
    assert M.moe_get_error() == M.MOE_OK
    rest = np.setdiff1d(np.arange(P), bad)
    for u, v in zip(*outs):
        np.testing.assert_array_equal(u[rest], v[rest])
    a, q, sf = outs[1]
    assert np.isnan(a[bad]).all() and np.isnan(sf[bad]).all() and (q[bad] == 0x7F).all()


@pytest.mark.parametrize("T,K", [(300, 1), (4, 2)])
def test_extreme_scales(T, K):
    """Rows from 2^-60 to 2^60 and zero rows: scales are taken whole, not as powers of two near them."""
    M = lib()
    c = _case(24, T, K, 2, 256, 128)
    c["x"] = bf16(c["x"] * np.exp2(np.linspace(-60, 20, c["P"]))[:, None])
    c["x"][1] = 0.0
    _check_products(M, c)


@pytest.mark.parametrize("T,K,E", [(300, 2, 4), (3, 2, 8)])
def test_data_gradient_products(T, K, E):
    """dy W2 and dH W1 as the plain product on the transposed weights."""
    M = lib()
    c = _case(25, T, K, E, 384, 256)
    P, h, F, offs = c["P"], c["h"], c["F"], c["offsets"]
    od = torch.from_numpy(offs.astype(np.int32)).cuda()
    rng = np.random.default_rng(26)
    for w, N, Kd in ((c["w2"], h, F), (c["w1"], 2 * F, h)):
        q, sf, qt, sft = u8(E, N, Kd), f32(E, N // 128, Kd // 128), u8(E, Kd, N), f32(E, Kd // 128, N // 128)
        M.moe_fp8_quantize_weights(E, N, Kd, to_dev(w, "bf16"), q, sf, qt, sft)
        dz = bf16(rng.standard_normal((P, N)))
        dq, dsf = quantize_dev(M, dz)
        out = torch.full((P, Kd), 33.0, dtype=torch.bfloat16, device="cuda")
        M.moe_expert_fc2_fp8(M.make_config(T, Kd, E, K, N), dq, dsf, od, qt, sft, out)
        W = X.dequantize(*X.quantize(w, True)).reshape(E, N, Kd).transpose(0, 2, 1).reshape(E * Kd, N)
        want, t = _z(X.dequantize(*X.quantize(dz)), offs, W, Kd, N)
        _near(out, want, t + 2.0 ** -8 * (np.abs(want) + t) + 1e-30)
    assert M.moe_get_error() == M.MOE_OK


def test_no_rows():
    M = lib()
    cfg = M.make_config(0, 128, 4, 2, 128)
    z8, zf = u8(4, 256, 128), f32(4, 2, 1)
    od = torch.zeros(5, dtype=torch.int32, device="cuda")
    e8, ef, eb = u8(1, 128), f32(1, 1), torch.full((1, 128), 33.0, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_fc1_fp8(cfg, e8, ef, od, None, z8, zf, None, eb, None, None)
    M.moe_expert_fc2_fp8(cfg, e8, ef, od, z8, zf, eb)
    M.moe_fp8_quantize(0, 128, None, None, None)
    assert torch.all(eb == 33.0) and M.moe_get_error() == M.MOE_OK


# ---- the path as it is used -------------------------------------------------------------
class Path:
    """Norm -> route -> dispatch in 8 bits -> FC1 -> FC2 -> combine, and the gradients
    that a training step takes back, on fixed buffers (so that it can be captured)."""

    def __init__(self, M, T, h, E, K, F, seed):
        self.M, self.T, self.h, self.E, self.K, self.F, self.P = M, T, h, E, K, F, T * K
        rng = np.random.default_rng(seed)
        self.w1 = bf16(rng.standard_normal((E * 2 * F, h)) / np.sqrt(h))
        self.w2 = bf16(rng.standard_normal((E * h, F)) / np.sqrt(F))
        self.w_r = to_dev(rng.standard_normal((E, h)) * 0.05, "f32")
        self.nw = to_dev(1 + 0.1 * rng.standard_normal(h), "f32")
        self.w1q, self.w1sf = weights_dev(M, self.w1, E)
        self.w2q, self.w2sf = weights_dev(M, self.w2, E)
        self.cfg = M.make_config(T, h, E, K, F)
        self.ws = torch.empty(M.moe_workspace_size(self.cfg), dtype=torch.uint8, device="cuda")
        self.nws = torch.empty(M.moe_rmsnorm_bwd_workspace_size(T, h), dtype=torch.uint8, device="cuda")
        P = self.P
        b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.x, self.res, self.sum, self.y, self.out = (b(T, h) for _ in range(5))
        self.q, self.sf, self.rstd = u8(T, h), f32(T, h // 128), f32(T)
        self.idx, self.prob = torch.zeros(T, K, dtype=torch.int32, device="cuda"), f32(T, K)
        self.maps = _maps(M, T, E, K)
        self.pq, self.psf = u8(P, h), f32(P, h // 128)
        self.save, self.aq, self.asf, self.yp = b(P, 2 * F), u8(P, F), f32(P, F // 128), b(P, h)
        self.dout, self.dyp, self.dprob = b(T, h), b(P, h), f32(T, K)
        self.dx, self.dnw = b(T, h), f32(h)

    def set(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (self.x, self.res, self.dout):
            t.normal_(generator=g)

    def step(self):
        M, m = self.M, self.maps
        M.moe_rmsnorm_fwd(self.T, self.h, M.MOE_BF16, self.x, self.res, self.nw, 1e-6, self.sum, self.y, self.q,
                          self.sf, self.rstd)
        M.moe_router_topk(self.cfg, self.y, self.w_r, None, None, None, self.idx, self.prob, ws=self.ws)
        M.moe_permute_fp8(self.cfg, self.q, self.sf, self.idx, self.prob, self.pq, self.psf, ws=self.ws, **m)
        M.moe_expert_fc1_fp8(self.cfg, self.pq, self.psf, m["offsets"], None, self.w1q, self.w1sf, self.save, None,
                             self.aq, self.asf)
        M.moe_expert_fc2_fp8(self.cfg, self.aq, self.asf, m["offsets"], self.w2q, self.w2sf, self.yp)
        M.moe_unpermute_combine(self.cfg, self.yp, m["dst_row"], self.prob, None, self.out)
        M.moe_unpermute_combine_bwd(self.cfg, self.dout, self.yp, m["dst_row"], self.prob, self.dyp, self.dprob)
        M.moe_rmsnorm_bwd(self.T, self.h, M.MOE_BF16, self.y, self.sum, self.rstd, self.nw, self.dout, self.dx,
                          self.dnw, self.nws)

    def outputs(self):
        return [self.sum, self.y, self.q, self.sf, self.idx, self.prob, *self.maps.values(), self.pq, self.psf,
                self.save, self.aq, self.asf, self.yp, self.out, self.dyp, self.dprob, self.dx, self.dnw]


@pytest.mark.parametrize("T,h,E,K,F", [(200, 512, 8, 2, 256), (5, 1024, 16, 4, 384)])
def test_path_step_by_step(T, h, E, K, F):
    """Each step of the path against the oracle on the step's own inputs."""
    M = lib()
    p = Path(M, T, h, E, K, F, seed=T)
    p.set(31)
    p.step()
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    n = lambda t: t.cpu().numpy() if t.dtype != torch.bfloat16 else to_np(t)  # noqa: E731
    v, yr, _ = X.rmsnorm(n(p.x), n(p.res), n(p.nw), 1e-6)
    d = 2.0 ** -16 * np.abs(yr)
    _near(p.y, yr, d + 2.0 ** -8 * (np.abs(yr) + d))
    sc = np.repeat(n(p.sf).astype(np.float64), 128, 1)
    deq = e4m3_decode(n(p.q)) * sc
    assert np.all(np.abs(deq - yr) <= d + np.maximum(2.0 ** -4 * np.abs(yr), 2.0 ** -10 * sc) * (1 + 2.0 ** -14))
    src, dst, offs = n(p.maps["src_token"]), n(p.maps["dst_row"]), n(p.maps["offsets"])
    np.testing.assert_array_equal(n(p.pq), n(p.q)[src])
    np.testing.assert_array_equal(n(p.psf), n(p.sf)[src])
    np.testing.assert_array_equal(offs, np.concatenate([[0], np.cumsum(np.bincount(n(p.idx).ravel(), minlength=E))]))
    W1, W2 = (X.dequantize(*X.quantize(w, True)) for w in (p.w1, p.w2))
    H, t = _z(deq[src], offs, W1, 2 * F, h)
    a_ref, da = _fc1_bound(H, t, np.ones(p.P))
    sa = np.repeat(n(p.asf).astype(np.float64), 128, 1)
    a = e4m3_decode(n(p.aq)) * sa
    assert np.all(np.abs(a - a_ref) <= da + np.maximum(2.0 ** -4 * (np.abs(a_ref) + da), 2.0 ** -10 * sa) * (1 + 2.0 ** -20))
    ypr, ty = _z(a, offs, W2, h, F)
    _near(p.yp, ypr, ty + 2.0 ** -8 * (np.abs(ypr) + ty) + 1e-30)
    out = X.combine(n(p.yp), dst, n(p.prob))
    S = X.combine(np.abs(n(p.yp)), dst, n(p.prob))
    _near(p.out, out, 2.0 ** -8 * np.abs(out) + 32 * U * S)
    dyp, dw = X.combine_bwd(n(p.dout), n(p.yp), dst, n(p.prob), np.zeros((p.P, h)))
    _near(p.dyp, dyp, (2.0 ** -8 + U) * np.abs(dyp))
    S = (np.abs(n(p.dout))[:, None, :] * np.abs(n(p.yp))[dst]).sum(2)
    _near(p.dprob, dw, (h / 128 + 16) * U * S)


def test_training_gradients_of_the_fp8_forward():
    """FC1's act_save and a, given to the bf16 backward with the combine's gradient: the
    expert gradients of the formula at those values (the backward's own tolerance)."""
    M = lib()
    c = _case(33, 160, 2, 4, 256, 256)
    c["x"] = bf16(np.random.default_rng(34).standard_normal((c["P"], 256)))
    P, E, h, F, offs = c["P"], c["E"], c["h"], c["F"], c["offsets"]
    cfg = M.make_config(c["T"], h, E, c["K"], F, flags=M.MOE_FLAG_RENORM | M.MOE_FLAG_SAVE_FOR_BWD)
    od = torch.from_numpy(offs.astype(np.int32)).cuda()
    xq, xsf = quantize_dev(M, c["x"])
    w1q, w1sf = weights_dev(M, c["w1"], E)
    save = torch.empty(P, 2 * F, dtype=torch.bfloat16, device="cuda")
    a = torch.empty(P, F, dtype=torch.bfloat16, device="cuda")
    pd = torch.from_numpy(c["p"]).cuda()
    M.moe_expert_fc1_fp8(cfg, xq, xsf, od, pd, w1q, w1sf, save, a, None, None)
    dy = bf16(np.random.default_rng(35).standard_normal((P, h)))
    ws = torch.empty(M.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    b = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    dx, dw1, dw2, dp = b(P, h), b(E, 2 * F, h), b(E, h, F), f32(P)
    w1, w2 = to_dev(c["w1"], "bf16").view(E, 2 * F, h), to_dev(c["w2"], "bf16").view(E, h, F)
    M.moe_grouped_mlp_bwd(cfg, to_dev(dy, "bf16"), to_dev(c["x"], "bf16"), save, a, od, pd, w1, w2, dx, dw1, dw2, dp, ws)
    assert M.moe_get_error() == M.MOE_OK
    H, av = to_np(save).astype(np.float64), to_np(a).astype(np.float64)
    for e in range(E):
        r = slice(offs[e], offs[e + 1])
        W1, W2 = c["w1"][e * 2 * F:(e + 1) * 2 * F], c["w2"][e * h:(e + 1) * h]
        g, u, pp = H[r, :F], H[r, F:], c["p"][r, None]
        sig = 1 / (1 + np.exp(-g))
        G = dy[r] @ W2
        dH = np.concatenate([pp * G * u * sig * (1 + g * (1 - sig)), pp * G * g * sig], 1)
        for got, want in ((dx[r], dH @ W1), (dw1[e], dH.T @ c["x"][r]), (dw2[e], dy[r].T @ av[r])):
            want = np.asarray(want)
            assert np.max(np.abs(to_np(got) - want)) <= 2e-2 * np.abs(want).max() + 1e-3


def test_path_captured_twice_and_replayed():
    """Two graphs of the path on two streams, each with its own buffers and workspace, replayed
    together on new inputs, against eager runs of the same inputs, bit for bit."""
    M = lib()
    paths = [Path(M, 150, 512, 8, 2, 256, 41), Path(M, 4, 1024, 16, 4, 256, 42)]
    streams = [torch.cuda.Stream() for _ in paths]
    graphs = []
    for p, s in zip(paths, streams):
        p.set(1)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            p.step()
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                p.step()
        graphs.append(g)
    for seed in (51, 52):
        for p in paths:
            p.set(seed)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in p.outputs()] for p in paths]
        for p, outs in zip(paths, got):
            p.step()
            torch.cuda.synchronize()
            for t, u in zip(p.outputs(), outs):
                assert torch.equal(t.view(torch.uint8), u.view(torch.uint8))
    assert M.moe_get_error() == M.MOE_OK


@pytest.mark.parametrize("T,K", [(100, 2), (3, 2)])
@pytest.mark.parametrize("offsets", [[5, -3, 900, 2, 7], [-10, 0, 10 ** 9, -(10 ** 9), 3], [0, 4, 4, 2, 6], [6, 6, 6, 6, 6]])
def test_offsets_outside_the_rows_are_kept_within_them(T, K, offsets):
    """Boundaries are taken between 0 and P and never before the one ahead of them."""
    M = lib()
    c = _case(61, T, K, 4, 256, 128)
    c["offsets"] = np.maximum.accumulate(np.clip(offsets, 0, c["P"]))
    want = _check_products(M, c)
    P, h, F = c["P"], c["h"], c["F"]
    cfg = M.make_config(T, h, 4, K, F)
    xq, xsf = quantize_dev(M, c["x"])
    w1q, w1sf = weights_dev(M, c["w1"], 4)
    a = torch.full((P, F), 33.0, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_fc1_fp8(cfg, xq, xsf, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                         torch.from_numpy(c["p"]).cuda(), w1q, w1sf, None, a, None, None)
    assert M.moe_get_error() == M.MOE_OK and torch.equal(a, want[1])


def test_strided_and_host_tensors_are_refused():
    M = lib()
    x = torch.zeros(128, 256, dtype=torch.bfloat16, device="cuda")
    q, sf = u8(128, 256), f32(128, 2)
    for bad in (x.t().contiguous().t(), x[:, :128], x.cpu()):
        with pytest.raises(ValueError):
            M.moe_fp8_quantize(128, 256, bad, q, sf)
    with pytest.raises(ValueError):
        M.moe_rmsnorm_fwd(128, 256, M.MOE_BF16, x, x.t().contiguous().t(), f32(256), 1e-6, y=x)


def test_large_offsets_of_bytes():
    """Rows whose byte offsets pass 2^31 and 2^32: the last rows are computed like the first."""
    M = lib()
    T, K, h, F = 300_000, 1, 16384, 128                    # 4.9e9 code bytes, 9.8e9 of bf16
    blk = bf16(np.random.default_rng(71).standard_normal((300, h)))
    x = to_dev(blk, "bf16").repeat(T // 300, 1)
    q, sf = torch.empty(T, h, dtype=torch.uint8, device="cuda"), torch.empty(T, h // 128, device="cuda")
    M.moe_fp8_quantize(T, h, x, q, sf)
    oq, osf = X.quantize(blk)
    for lo in (0, T // 2 // 300 * 300, T - 300):
        np.testing.assert_array_equal(q[lo:lo + 300].cpu().numpy(), oq)
        np.testing.assert_array_equal(sf[lo:lo + 300].cpu().numpy(), osf)
    w1 = bf16(np.random.default_rng(72).standard_normal((2 * F, h)) / 128)
    wq, wsf = weights_dev(M, w1, 1)
    cfg = M.make_config(T, h, 1, 1, F)
    a = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_fc1_fp8(cfg, q, sf, torch.tensor([0, T], dtype=torch.int32, device="cuda"), None, wq, wsf, None, a,
                         None, None)
    assert M.moe_get_error() == M.MOE_OK
    assert torch.equal(a[:300], a[-300:]) and torch.equal(a[:300], a[150_000:150_300])
    y, rq = torch.empty_like(x), torch.empty_like(q)
    M.moe_rmsnorm_fwd(T, h, M.MOE_BF16, x, None, torch.ones(h, device="cuda"), 1e-6, y=y, q=rq, sf=sf)
    assert torch.equal(y[:300], y[-300:]) and torch.equal(rq[:300], rq[-300:])
    dx, dw = torch.empty_like(x), torch.empty(h, device="cuda")
    r = torch.rand(300, device="cuda").repeat(T // 300)
    ws = torch.empty(M.moe_rmsnorm_bwd_workspace_size(T, h), dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm_bwd(T, h, M.MOE_BF16, y, x, r, torch.ones(h, device="cuda"), None, dx, dw, ws)
    assert torch.equal(dx[:300], dx[-300:])
    dst = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).view(T, 1).contiguous()
    M.moe_unpermute_combine_bwd(cfg, x, None, dst, None, y)
    assert torch.equal(y[:300], x[-300:].flip(0)) and torch.equal(y[-300:], x[:300].flip(0))
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    cws = torch.empty(M.moe_workspace_size(M.make_config(T, h, 1, 1, 8)), dtype=torch.uint8, device="cuda")
    M.moe_permute_fp8(M.make_config(T, h, 1, 1, 8), q, sf, idx, None, rq, torch.empty_like(sf), ws=cws, **_maps(M, T, 1, 1))
    assert M.moe_get_error() == M.MOE_OK and torch.equal(rq[-300:], q[-300:]) and torch.equal(rq[:300], q[:300])


@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_copies_and_other_streams(captured):
    """Calls that follow a copy, a fill and another stream's work (eager and in a graph), each
    reading what those wrote and overwriting what the one before read, many times over."""
    M = lib()
    rows, h, n = 700, 1024, 6
    g = torch.Generator(device="cuda").manual_seed(81)
    src = [torch.randn(rows, h, device="cuda", generator=g).bfloat16() for _ in range(n)]
    dst = torch.arange(rows, dtype=torch.int32, device="cuda").flip(0).view(rows, 1).contiguous()
    cfg = M.make_config(rows, h, 1, 1, 8)
    wt = torch.ones(h, device="cuda")
    x, y, z, res = (torch.zeros(rows, h, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    q, sf = u8(rows, h), f32(rows, h // 128)
    outs = [torch.zeros(rows, h, dtype=torch.bfloat16, device="cuda") for _ in range(n)]
    codes = [u8(rows, h) for _ in range(n)]
    main, other = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        for i in range(n):
            x.copy_(src[i])                                     # a copy, then a call that reads it
            M.moe_fp8_quantize(rows, h, x, q, sf)
            fork, join = torch.cuda.Event(), torch.cuda.Event()
            fork.record(main)
            other.wait_event(fork)
            with torch.cuda.stream(other):                      # another stream writes the residual
                res.copy_(src[(i + 1) % n])
                join.record(other)
            main.wait_event(join)
            M.moe_rmsnorm_fwd(rows, h, M.MOE_BF16, x, res, wt, 1e-6, x, y, q, sf)
            M.moe_unpermute_combine_bwd(cfg, y, None, dst, None, z)
            M.moe_unpermute_combine_bwd(cfg, z, None, dst, None, y)
            codes[i].copy_(q)
            outs[i].copy_(y)
            y.zero_()

    with torch.cuda.stream(main):
        if captured:
            work()
            main.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=main):
                work()
            for t in outs + codes:
                t.zero_()
            for _ in range(3):
                graph.replay()
        else:
            work()
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    for i in range(n):
        v, yw, qw, sw = src[i].clone(), torch.empty_like(x), u8(rows, h), f32(rows, h // 128)
        M.moe_rmsnorm_fwd(rows, h, M.MOE_BF16, v, src[(i + 1) % n], wt, 1e-6, None, yw, qw, sw)
        torch.cuda.synchronize()
        assert torch.equal(outs[i], yw) and torch.equal(codes[i], qw), i


@pytest.mark.parametrize("T,K", [(200, 2), (5, 2)])
def test_outputs_aligned_to_16_bytes_only(T, K):
    """Outputs on 16-byte boundaries that are not 32-byte ones: the same bits, nothing beside them."""
    M = lib()
    c = _case(91, T, K, 4, 384, 256)
    save, a, aq, asf, y = _check_products(M, c)
    P, E, h, F = c["P"], c["E"], c["h"], c["F"]
    cfg = M.make_config(T, h, E, K, F)
    od = torch.from_numpy(c["offsets"].astype(np.int32)).cuda()
    xq, xsf = quantize_dev(M, c["x"])
    w1q, w1sf = weights_dev(M, c["w1"], E)
    w2q, w2sf = weights_dev(M, c["w2"], E)

    def odd(like, skip):
        buf = torch.full((like.numel() + 64,), 7, dtype=like.dtype, device="cuda")
        view = buf[skip:skip + like.numel()].view(like.shape)
        assert view.data_ptr() % 32 == 16
        return buf, view

    bufs = {n: odd(t, 16 // t.element_size()) for n, t in dict(save=save, a=a, aq=aq, asf=asf, y=y).items()}
    v = {n: b[1] for n, b in bufs.items()}
    M.moe_expert_fc1_fp8(cfg, xq, xsf, od, torch.from_numpy(c["p"]).cuda(), w1q, w1sf, v["save"], v["a"], v["aq"], v["asf"])
    M.moe_expert_fc2_fp8(cfg, v["aq"], v["asf"], od, w2q, w2sf, v["y"])
    assert M.moe_get_error() == M.MOE_OK
    for n, want in dict(save=save, a=a, aq=aq, asf=asf, y=y).items():
        assert torch.equal(v[n], want), n
        skip = 16 // want.element_size()
        assert torch.all(bufs[n][0][:skip] == 7) and torch.all(bufs[n][0][skip + want.numel():] == 7)


@pytest.mark.parametrize("T,E", [(200, 8), (5000, 64)])
def test_permute_fp8_from_the_routers_histograms(T, E):
    """With MOE_FLAG_HIST_FROM_ROUTER the maps start from what the router left in the workspace."""
    M = lib()
    h, K = 256, 2
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, h, device="cuda", generator=g).bfloat16()
    w_r = torch.randn(E, h, device="cuda", generator=g) * 0.05
    q, sf = u8(T, h), f32(T, h // 128)
    got = []
    for flags in (M.MOE_FLAG_RENORM, M.MOE_FLAG_RENORM | M.MOE_FLAG_HIST_FROM_ROUTER):
        cfg = M.make_config(T, h, E, K, 128, flags=flags)
        ws = torch.empty(M.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        idx, prob = torch.empty(T, K, dtype=torch.int32, device="cuda"), f32(T, K)
        M.moe_fp8_quantize(T, h, x, q, sf)
        M.moe_router_topk(cfg, x, w_r, None, None, None, idx, prob, ws=ws)
        m, pq, psf = _maps(M, T, E, K), u8(T * K, h), f32(T * K, h // 128)
        M.moe_permute_fp8(cfg, q, sf, idx, prob, pq, psf, ws=ws, **m)
        got.append([idx, prob, pq, psf, *m.values()])
    assert M.moe_get_error() == M.MOE_OK
    for a, b in zip(*got):
        assert torch.equal(a, b)
