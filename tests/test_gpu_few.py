"""GPU parity of moe_layer_fwd_few and moe_layer_fwd_few_mxfp4 (the layer for a
few tokens) against the float64 oracle.

Tolerance of y, from the roundings on the way (all sums fp32, u = 2^-23 an
addition, of n terms n u sum|terms|): FC1's sums, carried through the
activation (|phi'| <= 1.13; the expert's hidden values are then two bf16 numbers,
the second what the first left: at most 2^-8 2^-8 |a|; with many tokens an expert
one number, 2^-8 |a|), FC2's sums, p (relative 2^-18, the router's logits
included) and the bf16 y, 2^-8 |y|.  The bound is evaluated per element from the
absolute values of the same products.  Beside MXFP4 weights tokens and hidden
values are sums of four E2M1 blocks of 32 columns: part 0 rounds to steps of at
most s (s the power of two with the block's largest value in [2 s, 4 s)) and leaves
at most s / 2, which is 2 units of part 1's scale s / 4, where E2M1's steps are at
most 1/2; so it leaves s / 16 = 2 units of s / 32, part 2 s / 128 = 2 units of
s / 256, part 3 s / 1024, at most 2^-11 of the block's largest value."""

import numpy as np
import pytest
import torch

from gpu_util import check_routing, lib, needs_gpu, to_dev, to_np
from oracle import moe_oracle as O
from oracle import mxfp4_oracle as X4

pytestmark = [pytest.mark.gpu, needs_gpu]

U = 2.0 ** -23


def bf16(a):
    return to_np(torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16))


class Few:
    """Host inputs, device tensors and the float64 result with its bound."""

    def __init__(self, T, h, E, K, F, seed=0, score=0, act=1, bias=False, shared=0, sel=False,
                 gate=False, renorm=True, force=False, capacity=0, mx=False, x=None):
        rng = np.random.default_rng(seed + 1000 * T + h)
        self.__dict__.update(locals())
        r1 = 2 * F if act == 1 else F
        drawn = rng.standard_normal((T, h))          # drawn in any case: the weights do not depend on x
        self.x = bf16(drawn if x is None else x)
        self.w_r = (rng.standard_normal((E, h)) / np.sqrt(h)).astype(np.float32)
        self.gb = rng.standard_normal(E).astype(np.float32) if gate else None
        self.sb = (0.1 * rng.standard_normal(E)).astype(np.float32) if sel else None
        mat = lambda n, r, c: bf16(rng.standard_normal((n, r, c)) / np.sqrt(c))  # noqa: E731
        self.w1, self.w2 = mat(E, r1, h), mat(E, h, F)
        self.b1 = bf16(rng.standard_normal((E, F)) / np.sqrt(h)) if bias else None
        self.b2 = bf16(rng.standard_normal((E, h)) / np.sqrt(F)) if bias else None
        self.w1s, self.w2s = (mat(1, r1, h)[0], mat(1, h, F)[0]) if shared else (None, None)
        if mx:  # the values of the 4-bit weights
            for n in ("w1", "w2", "w1s", "w2s"):
                w = getattr(self, n)
                if w is not None:
                    v = X4.dequantize(*X4.quantize(w.reshape(-1, w.shape[-1]))).reshape(w.shape)
                    setattr(self, n + "_bf16", w)
                    setattr(self, n, v)

    def cfg(self, M, extra=0):
        f = (M.MOE_FLAG_RENORM if self.renorm else 0) | (M.MOE_FLAG_FORCE_BALANCE if self.force else 0)
        return M.make_config(self.T, self.h, self.E, self.K, self.F, M.MOE_BF16, self.score, self.act,
                             int(self.bias), self.shared, f | extra, capacity=self.capacity)

    def device(self, M):
        d = {"x": to_dev(self.x, "bf16"), "w_r": to_dev(self.w_r, "f32")}
        for n in ("gb", "sb"):
            d[n] = None if getattr(self, n) is None else to_dev(getattr(self, n), "f32")
        for n in ("b1", "b2"):
            d[n] = None if getattr(self, n) is None else to_dev(getattr(self, n), "bf16")
        for n in ("w1", "w2", "w1s", "w2s"):
            w = getattr(self, n)
            if w is None:
                d[n] = d[n + "_sf"] = None
            elif not self.mx:
                d[n] = to_dev(w, "bf16")
            else:
                w = getattr(self, n + "_bf16")
                cols, groups = w.shape[-1], (w.shape[0] if w.ndim == 3 else 1)
                rows = w.size // cols
                d[n] = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
                d[n + "_sf"] = torch.zeros(M.moe_mxfp8_scale_bytes(rows, cols, groups),
                                           dtype=torch.uint8, device="cuda")
                M.moe_mxfp4_quantize(rows, cols, groups, None, to_dev(w.reshape(rows, cols), "bf16"),
                                     d[n], d[n + "_sf"])
        self.d = d
        self.ws = torch.full((M.moe_workspace_size(self.cfg(M)),), 0xA5, dtype=torch.uint8, device="cuda")
        self.y = torch.full((self.T, self.h), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.idx = torch.full((self.T, self.K), -1, dtype=torch.int32, device="cuda")
        self.prob = torch.full((self.T, self.K), -1.0, device="cuda")
        return self

    def call(self, M, y=None, idx=True, ws=None, stream=None):
        d, y, ws = self.d, self.y if y is None else y, self.ws if ws is None else ws
        i, p = (self.idx, self.prob) if idx else (None, None)
        if self.mx:
            M.moe_layer_fwd_few_mxfp4(self.cfg(M), d["x"], d["w_r"], d["gb"], d["sb"], d["w1"],
                                      d["w1_sf"], d["w2"], d["w2_sf"], d["w1s"], d["w1s_sf"],
                                      d["w2s"], d["w2s_sf"], y, i, p, ws, stream)
        else:
            M.moe_layer_fwd_few(self.cfg(M), d["x"], d["w_r"], d["gb"], d["sb"], d["w1"], d["b1"],
                                d["w2"], d["b2"], d["w1s"], d["w2s"], y, i, p, ws, stream)

    def expert(self, x, w1, w2, b1, b2):
        """(output, its bound) of one expert on rows x."""
        F, h = self.F, self.h
        z = x @ w1.T + (0 if b1 is None else b1)
        dz = h * U * (np.abs(x) @ np.abs(w1).T + (0 if b1 is None else np.abs(b1)))

        def parts(v):  # what a block's four parts leave
            m = np.abs(v).reshape(len(v), -1, 32).max(2)
            return 2.0 ** -11 * np.repeat(m, 32, axis=1)

        if self.mx:
            dz = dz + parts(x) @ np.abs(w1).T
        if self.act == 1:
            g, u, dg, du = z[:, :F], z[:, F:], dz[:, :F], dz[:, F:]
            a = O.silu(g) * u
            da = 1.13 * dg * (np.abs(u) + du) + (np.abs(O.silu(g)) + 1.13 * dg) * du
        else:
            a, da = O.gelu(z), 1.13 * dz
        da = da + 2.0 ** -18 * (np.abs(a) + da)
        many = self.T > 8 and self.T * self.K > 4 * self.E
        da = da + (parts(np.abs(a) + da) if self.mx else 2.0 ** (-8 if many else -16) * (np.abs(a) + da))
        o = a @ w2.T + (0 if b2 is None else b2)
        S = np.abs(a) @ np.abs(w2).T
        return o, da @ np.abs(w2).T + F * U * S

    def check(self, M):
        T, K = self.T, self.K
        logits = O.gating_logits(self.x, self.w_r, self.gb)
        ridx, rprob = O.route(logits, K, self.score, self.renorm, self.sb, self.force)
        gidx, gprob = to_np(self.idx), to_np(self.prob)
        ok = check_routing(gidx, gprob, ridx, rprob, logits, K, self.score, self.sb, self.force) \
            if T > 60 or self.force else None
        if ok is None:  # few tokens: a share of them says nothing, each is looked at
            m = O.selection_margin(logits, K, self.score, self.sb) >= 1e-5
            m &= O.order_margin(logits, K, self.score, self.sb) >= 1e-5
            np.testing.assert_array_equal(gidx[m], ridx[m])
            np.testing.assert_allclose(gprob[m], rprob[m], rtol=1e-5, atol=1e-6)
            ok = np.array([sorted(gidx[t]) == sorted(ridx[t]) for t in range(T)])
            assert ok[m].all()
        y, tol = np.zeros((T, self.h)), np.zeros((T, self.h))
        x = self.x.astype(np.float64)
        seen = {}
        for t in range(T):
            for k in range(K):
                e = int(gidx[t, k])
                seen[e] = seen.get(e, 0) + 1
                if self.capacity and seen[e] > self.capacity:
                    continue
                o, do = self.expert(x[t:t + 1], self.w1[e].astype(np.float64),
                                    self.w2[e].astype(np.float64),
                                    None if self.b1 is None else self.b1[e].astype(np.float64),
                                    None if self.b2 is None else self.b2[e].astype(np.float64))
                p = float(gprob[t, k])
                y[t] += p * o[0]
                tol[t] += p * (do[0] + 2.0 ** -18 * np.abs(o[0]))
        if self.shared:
            o, do = self.expert(x, self.w1s.astype(np.float64), self.w2s.astype(np.float64), None, None)
            y += o
            tol += do
        tol += 2.0 ** -8 * (np.abs(y) + tol) + 1e-30
        err = np.abs(to_np(self.y).astype(np.float64) - y)
        assert np.all(err <= tol), float((err / tol).max())
        # and as a whole: two 16-bit roundings (hidden values, y) of relative
        # size 2^-8 at most leave a norm far below a percent
        assert np.linalg.norm(err) <= 0.008 * np.linalg.norm(y) + 1e-30


def run(**kw):
    M = lib()
    f = Few(**kw).device(M)
    f.call(M)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    f.check(M)
    return f


BF16 = [
    dict(T=1, h=64, E=8, K=2, F=64),
    dict(T=1, h=2048, E=64, K=8, F=256),
    dict(T=2, h=8, E=4, K=1, F=8),                                   # the smallest rows
    dict(T=3, h=520, E=16, K=3, F=136, score=1, sel=True, shared=1),
    dict(T=5, h=1032, E=256, K=8, F=72, score=1, sel=True, shared=1),
    dict(T=7, h=264, E=5, K=2, F=1000, act=0, bias=True),
    dict(T=8, h=512, E=3, K=3, F=264, act=0),
    dict(T=11, h=296, E=6, K=3, F=200, act=0, bias=True, shared=1),
    dict(T=9, h=256, E=1, K=1, F=520, gate=True),                    # one expert has every token
    dict(T=16, h=1024, E=8, K=2, F=512, shared=1),
    dict(T=17, h=776, E=100, K=16, F=88, renorm=False, score=1),
    dict(T=31, h=384, E=8, K=8, F=128, renorm=False),                # every expert, every token
    dict(T=33, h=640, E=2, K=1, F=384),
    dict(T=64, h=512, E=1, K=1, F=256, shared=1),                    # 64 rows in one expert
    dict(T=64, h=1024, E=32, K=6, F=320),
    dict(T=63, h=136, E=9, K=4, F=5008),                             # long second projection
    dict(T=12, h=256, E=8, K=2, F=128, force=True),
    dict(T=40, h=256, E=4, K=2, F=128, capacity=7, shared=1),        # drops
    dict(T=50, h=128, E=8, K=2, F=136, capacity=1),
    dict(T=64, h=1032, E=256, K=8, F=16),                            # a router warp with 8 tokens,
    dict(T=37, h=1024, E=120, K=4, F=24, score=1),                   # 4
    dict(T=23, h=2048, E=64, K=8, F=40, sel=True),                   # and 2
]
MX = [
    dict(T=1, h=128, E=8, K=2, F=128),
    dict(T=1, h=2048, E=64, K=8, F=256, score=1, sel=True, shared=1),
    dict(T=2, h=640, E=4, K=1, F=384),
    dict(T=5, h=1152, E=256, K=8, F=128, score=1, sel=True, shared=1),
    dict(T=8, h=1024, E=1, K=1, F=640),
    dict(T=13, h=512, E=8, K=2, F=1024, gate=True),
    dict(T=33, h=384, E=3, K=2, F=256, renorm=False),
    dict(T=64, h=256, E=2, K=2, F=512, shared=1),
    dict(T=64, h=1024, E=32, K=6, F=384),
    dict(T=40, h=256, E=4, K=2, F=128, capacity=7),
    dict(T=20, h=128, E=16, K=4, F=128, force=True),
]


def _id(c):
    return "_".join(f"{k}{v}" for k, v in c.items())


@pytest.mark.parametrize("c", BF16, ids=_id)
def test_bf16_weights(c):
    run(**c)


@pytest.mark.parametrize("c", MX, ids=_id)
def test_mxfp4_weights(c):
    run(mx=True, **c)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 40])
def test_token_magnitudes(mx, scale):
    """Tokens far from 1, beside ordinary ones, and an outlier in a row; the
    activation's product must stay finite."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 256))
    x[1] *= scale
    x[3, 7] *= 1e4                                   # one outlier in a row
    run(T=4, h=256, E=4, K=2, F=128, mx=mx, x=x, force=True)


@pytest.mark.parametrize("mx", [False, True])
def test_non_finite_tokens_stay_in_their_rows(mx):
    M = lib()
    kw = dict(T=9, h=256, E=4, K=2, F=128, mx=mx, force=True, seed=3)
    clean = run(**kw)
    x = clean.x.copy()
    x[2, 5], x[6, 100], x[7, 0] = np.nan, np.inf, -np.inf
    f = Few(**dict(kw, x=x)).device(M)
    f.call(M)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    rest = [0, 1, 3, 4, 5, 8]
    assert torch.equal(f.y[rest], clean.y[rest])
    assert not torch.isfinite(f.y[[2, 6, 7]].float()).any()


@pytest.mark.parametrize("mx", [False, True])
def test_reruns_outputs_alone_and_equal_tokens(mx):
    """Bitwise the same on a dirty workspace, with and without the routing
    outputs; equal tokens get equal rows; nothing is written past y."""
    M = lib()
    rng = np.random.default_rng(11)
    x = np.repeat(rng.standard_normal((3, 384)), [10, 1, 9], axis=0)
    f = run(T=20, h=384, E=8, K=3, F=256, mx=mx, x=x, shared=1)
    guard = torch.full((22, 384), 7.0, dtype=torch.bfloat16, device="cuda")
    f.call(M, y=guard[:20], idx=False)
    torch.cuda.synchronize()
    assert torch.equal(guard[:20], f.y) and (guard[20:] == 7).all()
    assert torch.equal(f.y[0], f.y[9]) and torch.equal(f.y[11], f.y[19])


@pytest.mark.parametrize("mx", [False, True])
def test_side_stream_graphs_and_two_at_once(mx):
    """A captured call replayed on new tokens; two calls in flight on two
    streams, each with its own workspace; two graphs one after the other on one."""
    M = lib()
    f = run(T=6, h=512, E=16, K=4, F=256, mx=mx, shared=1)
    want = f.y.clone()
    g = Few(T=37, h=384, E=8, K=2, F=128, mx=mx).device(M)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        f.call(M, stream=s1)
        g.call(M, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(f.y, want)
    g.check(M)
    other = g.y.clone()
    big = torch.empty(max(f.ws.numel(), g.ws.numel()), dtype=torch.uint8, device="cuda").fill_(0x3C)
    graphs = []
    for c in (f, g):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.call(M, ws=big)
        graphs.append(gr)
    x0 = f.d["x"].clone()
    f.d["x"].copy_(-x0)
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(g.y, other) and not torch.equal(f.y, want)
    f.d["x"].copy_(x0)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(f.y, want)
    assert M.moe_get_error() == M.MOE_OK


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E", [8, 64, 256])
def test_equal_logits_pick_the_lowest_experts(E, score):
    """Experts with the same router row have the same logit to the bit."""
    M = lib()
    f = Few(T=6, h=256, E=E, K=4, F=64, score=score, seed=4)
    f.w_r[:] = f.w_r[0]
    f.device(M).call(M)
    torch.cuda.synchronize()
    assert (f.idx.cpu() == torch.arange(4, dtype=torch.int32)).all()
    assert (f.prob == 0.25).all()
    f = Few(T=6, h=256, E=E, K=4, F=64, score=score, seed=4)
    f.w_r[E // 2:] = f.w_r[:E - E // 2]              # every expert of the lower half again
    f.device(M).call(M)
    torch.cuda.synchronize()
    idx, half = to_np(f.idx).astype(int), E // 2
    for row in idx:                                  # a pair's lower one is next to its upper one
        for k in (0, 2):
            if row[k] < half:
                assert row[k + 1] == row[k] + half
    assert M.moe_get_error() == M.MOE_OK


@pytest.mark.parametrize("mx", [False, True])
def test_routed_non_finite_tokens(mx):
    """Tokens whose logits are NaN take some K different experts and stay NaN; the
    others are as without them."""
    M = lib()
    kw = dict(T=9, h=256, E=40, K=5, F=128, mx=mx, seed=3)
    clean = run(**kw)
    x = clean.x.copy()
    x[2, 5], x[6, 100] = np.nan, np.inf
    f = Few(**dict(kw, x=x)).device(M)
    f.call(M)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    idx = to_np(f.idx).astype(int)
    assert all(len(set(r)) == 5 and min(r) >= 0 and max(r) < 40 for r in idx)
    rest = [0, 1, 3, 4, 5, 7, 8]
    assert torch.equal(f.y[rest], clean.y[rest]) and torch.equal(f.idx[rest], clean.idx[rest])
    assert torch.isnan(f.y[2].float()).all()


def test_agrees_with_the_layer_pass():
    """moe_layer_fwd on the same inputs: the same routing, outputs within the
    bf16 roundings of the two (relative norm below a percent)."""
    M = lib()
    f = run(T=48, h=1024, E=16, K=4, F=512, shared=1, score=1, sel=True)
    cfg, d = f.cfg(M), f.d
    y, idx = torch.empty_like(f.y), torch.empty_like(f.idx)
    M.moe_layer_fwd(cfg, d["x"], d["w_r"], None, d["sb"], d["w1"], None, d["w2"], None, d["w1s"],
                    d["w2s"], y, idx, None, f.ws)
    torch.cuda.synchronize()
    assert torch.equal(idx, f.idx)
    assert (y.float() - f.y.float()).norm() <= 0.01 * y.float().norm()


def test_mxfp4_set_as_a_server_uses_it():
    """Weights quantised once serve both a large batch (dispatch, quantised
    rows, the grouped products, combine) and a few tokens; the two differ only
    by the 4-bit rounding of the large batch's activations."""
    M = lib()
    few = run(T=8, h=512, E=8, K=2, F=256, mx=True, seed=21)
    T, h, E, K, F = 8, 512, 8, 2, 256
    cfg = M.make_config(T, h, E, K, F)
    P, d = T * K, few.d
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets, dst = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T, K, **i32)
    src, pp = torch.empty(P, **i32), torch.empty(P, device="cuda")
    xp = torch.empty(P, h, dtype=torch.bfloat16, device="cuda")
    M.moe_permute(cfg, d["x"], few.idx, few.prob, xp, counts, offsets, dst, src, pp, few.ws)
    u8 = dict(dtype=torch.uint8, device="cuda")
    xq, xsf = torch.empty(P, h // 2, **u8), torch.empty(M.moe_mxfp8_scale_bytes(P, h, E), **u8)
    aq, asf = torch.empty(P, F // 2, **u8), torch.empty(M.moe_mxfp8_scale_bytes(P, F, E), **u8)
    M.moe_mxfp4_quantize(P, h, E, offsets, xp, xq, xsf)
    M.moe_expert_fc1_mxfp4(cfg, xq, xsf, offsets, pp, d["w1"], d["w1_sf"], None, aq, asf)
    yp, y = torch.empty_like(xp), torch.empty(T, h, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_fc2_mxfp4(cfg, aq, asf, offsets, d["w2"], d["w2_sf"], yp)
    M.moe_unpermute_combine(cfg, yp, dst, None, None, y)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    # E2M1's steps are at most a quarter of the value: two such roundings
    # (x and a) stay below the sum of both, as norms
    assert (y.float() - few.y.float()).norm() <= 0.5 * few.y.float().norm()
    assert (y.float() - few.y.float()).norm() > 0


@pytest.mark.parametrize("mx", [False, True])
def test_nothing_is_written_outside_the_buffers(mx):
    """The workspace and every output between guard bytes; dirty inside."""
    M = lib()
    for kw in (dict(T=1, h=128, E=8, K=2, F=128), dict(T=33, h=640, E=7, K=5, F=384, shared=1),
               dict(T=64, h=256, E=256, K=16, F=256, force=True)):
        f = Few(mx=mx, seed=31, **kw).device(M)
        n, G = f.ws.numel(), 8192
        big = torch.full((n + 2 * G,), 0x5A, dtype=torch.uint8, device="cuda")
        y = torch.full((f.T + 8, f.h), 3.0, dtype=torch.bfloat16, device="cuda")
        idx = torch.full((f.T + 8, f.K), -7, dtype=torch.int32, device="cuda")
        prob = torch.full((f.T + 8, f.K), -7.0, device="cuda")
        f.idx, f.prob, f.y = idx[4:-4], prob[4:-4], y[4:-4]
        # rows of 2 * 128 bytes and more keep y's first row 16-byte aligned
        f.call(M, ws=big[G:G + n])
        torch.cuda.synchronize()
        assert M.moe_get_error() == M.MOE_OK
        assert (big[:G] == 0x5A).all() and (big[G + n:] == 0x5A).all()
        for b, v in ((y, 3.0), (idx, -7), (prob, -7.0)):
            assert (b[:4] == v).all() and (b[-4:] == v).all()
        f.check(M)


def test_mxfp4_blocks_of_nan_and_zero_scales():
    """A weight block of NaN scale makes its output columns NaN, for the tokens of
    its expert alone; a block of zeros (scale code 0) adds nothing."""
    M = lib()
    f = Few(T=6, h=256, E=3, K=1, F=128, mx=True, force=True, seed=5)
    w2 = f.w2_bf16.copy()
    w2[1, 40, 64:96] = np.nan          # expert 1 (tokens 1 and 4), output column 40
    w2[2, 7, 32:64] = 0.0
    f.w2_bf16, clean = w2, f.w2.copy()
    clean[1, 40, 64:96] = 0.0
    clean[2, 7, 32:64] = 0.0
    f.w2 = clean
    f.device(M)
    f.call(M)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    y = to_np(f.y)
    nan = np.isnan(y)
    assert nan[[1, 4], 40].all() and nan.sum() == 2
    f.y = torch.where(torch.isnan(f.y), torch.zeros_like(f.y), f.y)
    keep = np.ones((6, 256), bool)
    keep[[1, 4], 40] = False
    ref, tol = np.zeros((6, 256)), np.zeros((6, 256))
    for t in range(6):
        o, do = f.expert(f.x[t:t + 1].astype(np.float64), f.w1[t % 3], f.w2[t % 3], None, None)
        ref[t], tol[t] = o[0], do[0]
    tol += 2.0 ** -8 * (np.abs(ref) + tol)
    assert (np.abs(to_np(f.y) - ref) <= tol)[keep].all()


def test_in_place_and_long_rows():
    """y may be x; a long second projection takes several slices of F."""
    M = lib()
    f = run(T=3, h=512, E=2, K=1, F=9000)
    want = f.y.clone()
    f.call(M, y=f.d["x"])
    torch.cuda.synchronize()
    assert torch.equal(f.d["x"], want)


def test_injected_failure_enqueues_nothing():
    M = lib()
    f = Few(T=4, h=128, E=4, K=2, F=128).device(M)
    assert M.moe_test_inject_cuda_failure(1) == 0
    with pytest.raises(M.MoeError) as e:
        f.call(M)
    assert e.value.status == M.MOE_ERR_CUDA
    torch.cuda.synchronize()
    assert torch.isnan(f.y).all() and (f.idx == -1).all()
    f.call(M)
    torch.cuda.synchronize()
    f.check(M)
