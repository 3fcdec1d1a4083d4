"""GPU parity of moe_rmsnorm_fwd / moe_rmsnorm_bwd against the float64 oracle.

Tolerances (U = 2^-24, half a step of fp32; eps/2 of a type where an output is
rounded to it).  A sum of h values passes at most 160 additions one after the
other (at most 64 values a thread, 5 shuffles, at most 32 warps, with room for
another split), each off by U of the sum of magnitudes.  v is one rounding.
r = 1 / sqrt(ss / h + eps): half the relative error of ss (160 + 2 roundings) and
4 more: 85 U <= 2^-17.  y adds 3 roundings.  The mean of g n is within 170 U of
the mean of |g n|; dx carries it times r |n|, and 6 roundings of each term.  dw
sums one product a row through at most rows + 512 additions."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu, to_dev, to_np
from oracle import fp8_oracle as X
from oracle.mxfp8_oracle import e4m3_decode

pytestmark = [pytest.mark.gpu, needs_gpu]

U = 2.0 ** -24
EPS = 1e-6
HALF = {"bf16": 2.0 ** -8, "f32": U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rounded(a, dtype):
    t = torch.from_numpy(np.asarray(a, np.float32))
    return (t.to(torch.bfloat16) if dtype == "bf16" else t).float().numpy()


def _inputs(rows, h, dtype, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    x, res = (rounded(scale * s * rng.standard_normal((rows, h)), dtype) for s in (1.0, 2.0))
    return x, res, (1 + 0.1 * rng.standard_normal(h)).astype(np.float32)


def check_fwd(x, res, w, dtype, sum=None, y=None, q=None, sf=None, rstd=None):
    v, yr, r = X.rmsnorm(x, res, w, EPS)
    if sum is not None:
        assert np.all(np.abs(to_np(sum) - v) <= (HALF[dtype] + 2 * U) * np.abs(v))
    if rstd is not None:
        assert np.all(np.abs(to_np(rstd) - r) <= 2.0 ** -17 * r)
    d = (2.0 ** -17 + 4 * U) * np.abs(yr)
    if y is not None:
        assert np.all(np.abs(to_np(y) - yr) <= d + HALF[dtype] * (np.abs(yr) + d))
    if q is not None:
        s = sf.cpu().numpy().astype(np.float64)
        top = np.abs(yr).reshape(s.shape + (128,)).max(2)
        assert np.all(np.abs(s * 448 - top) <= (2.0 ** -17 + 8 * U) * top)
        sc = np.repeat(s, 128, 1)
        err = np.abs(e4m3_decode(q.cpu().numpy()) * sc - yr)
        assert np.all(err <= d + np.maximum(2.0 ** -4 * np.abs(yr), 2.0 ** -10 * sc) * (1 + 2.0 ** -14))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,h", [(1, 128), (7, 7168), (33, 2048), (5, 256), (3, 8320), (2, 16384), (1, 65536),
                                    (1021, 384), (130, 4096), (4, 640)])
def test_forward(rows, h, dtype):
    M = lib()
    x, res, w = _inputs(rows, h, dtype, rows + h)
    xd, rd, wd = to_dev(x, dtype), to_dev(res, dtype), to_dev(w, "f32")
    e = lambda *s, dt=DT[dtype]: torch.full(s, 77, dtype=dt, device="cuda")  # noqa: E731
    o = dict(sum=e(rows, h), y=e(rows, h), q=e(rows, h, dt=torch.uint8), sf=e(rows, h // 128, dt=torch.float32),
             rstd=e(rows, dt=torch.float32))
    dt = M.MOE_BF16 if dtype == "bf16" else M.MOE_F32
    M.moe_rmsnorm_fwd(rows, h, dt, xd, rd, wd, EPS, **o)
    check_fwd(x, res, w, dtype, **o)
    # each output alone is the same bits; without a residual
    y2, q2, sf2 = e(rows, h), e(rows, h, dt=torch.uint8), e(rows, h // 128, dt=torch.float32)
    M.moe_rmsnorm_fwd(rows, h, dt, xd, rd, wd, EPS, y=y2)
    M.moe_rmsnorm_fwd(rows, h, dt, xd, rd, wd, EPS, q=q2, sf=sf2)
    assert torch.equal(y2, o["y"]) and torch.equal(q2, o["q"]) and torch.equal(sf2, o["sf"])
    M.moe_rmsnorm_fwd(rows, h, dt, xd, None, wd, EPS, o["sum"], y2, q2, sf2, o["rstd"])
    check_fwd(x, None, w, dtype, o["sum"], y2, q2, sf2, o["rstd"])
    assert torch.equal(o["sum"], xd)


@pytest.mark.parametrize("dtype,h", [("bf16", 8), ("bf16", 1000), ("bf16", 2056), ("f32", 4), ("f32", 1004),
                                     ("f32", 2052), ("f32", 36)])
def test_forward_and_backward_of_odd_widths(dtype, h):
    M = lib()
    rows = 19
    x, res, w = _inputs(rows, h, dtype, h)
    pad = torch.full((rows * h + 64,), 55.0, dtype=DT[dtype], device="cuda")  # what lies behind the last row
    y = pad[:rows * h].view(rows, h)
    rstd = torch.empty(rows, device="cuda")
    dt = M.MOE_BF16 if dtype == "bf16" else M.MOE_F32
    M.moe_rmsnorm_fwd(rows, h, dt, to_dev(x, dtype), to_dev(res, dtype), to_dev(w, "f32"), EPS, y=y, rstd=rstd)
    check_fwd(x, res, w, dtype, y=y, rstd=rstd)
    assert torch.all(pad[rows * h:] == 55.0)
    _check_bwd(M, rows, h, dtype, True, h)


def test_forward_in_place():
    """The sum in x's or res's buffer, y in x's."""
    M = lib()
    x, res, w = _inputs(50, 1024, "bf16", 5)
    wd = to_dev(w, "f32")
    want_s, want_y = torch.empty(2, 50, 1024, dtype=torch.bfloat16, device="cuda").unbind()
    M.moe_rmsnorm_fwd(50, 1024, M.MOE_BF16, to_dev(x, "bf16"), to_dev(res, "bf16"), wd, EPS, want_s, want_y)
    xd, rd = to_dev(x, "bf16"), to_dev(res, "bf16")
    M.moe_rmsnorm_fwd(50, 1024, M.MOE_BF16, xd, rd, wd, EPS, rd, xd)
    assert torch.equal(rd, want_s) and torch.equal(xd, want_y)
    xd, rd = to_dev(x, "bf16"), to_dev(res, "bf16")
    M.moe_rmsnorm_fwd(50, 1024, M.MOE_BF16, xd, rd, wd, EPS, xd, want_s)
    assert torch.equal(want_s, want_y)


def test_zero_large_and_non_finite_rows():
    """A row of zeros gives zeros (eps > 0); rows with a NaN are NaN and leave the others alone."""
    M = lib()
    x, res, w = _inputs(6, 512, "bf16", 6)
    x[1], res[1] = 0.0, 0.0
    x[4, 9] = np.nan
    x[2] = rounded(x[2] * 2.0 ** 40, "bf16")
    y = torch.empty(6, 512, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(6, 512, dtype=torch.uint8, device="cuda")
    sf = torch.empty(6, 4, device="cuda")
    M.moe_rmsnorm_fwd(6, 512, M.MOE_BF16, to_dev(x, "bf16"), to_dev(res, "bf16"), to_dev(w, "f32"), EPS, y=y, q=q, sf=sf)
    rest = [0, 1, 2, 3, 5]
    check_fwd(x[rest], res[rest], w, "bf16", y=y[rest])
    assert torch.all(y[1] == 0) and torch.all((q[1] & 127) == 0) and torch.all(sf[1] == 2.0 ** -125)
    assert torch.isnan(y[4]).all() and torch.isnan(sf[4]).all() and torch.all(q[4] == 0x7F)


def _check_bwd(M, rows, h, dtype, with_dsum, seed):
    rng = np.random.default_rng(seed)
    v = rounded(2 * rng.standard_normal((rows, h)), dtype)
    dy, ds = (rounded(rng.standard_normal((rows, h)), dtype) for _ in range(2))
    w = (1 + 0.1 * rng.standard_normal(h)).astype(np.float32)
    r = (1 / np.sqrt((v.astype(np.float64) ** 2).mean(1) + EPS)).astype(np.float32)
    ds = ds if with_dsum else None
    dt = M.MOE_BF16 if dtype == "bf16" else M.MOE_F32
    dev = dict(dy=to_dev(dy, dtype), sum=to_dev(v, dtype), rstd=to_dev(r, "f32"), w=to_dev(w, "f32"),
               dsum=to_dev(ds, dtype) if with_dsum else None)
    dx = torch.full((rows, h), 77.0, dtype=DT[dtype], device="cuda")
    dw = torch.full((h,), 77.0, device="cuda")
    ws = torch.empty(M.moe_rmsnorm_bwd_workspace_size(rows, h), dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm_bwd(rows, h, dt, dev["dy"], dev["sum"], dev["rstd"], dev["w"], dev["dsum"], dx, dw, ws)
    rx, rw = X.rmsnorm_bwd(dy, v, r, w, ds)
    n = np.abs(v.astype(np.float64)) * r[:, None]
    g = np.abs(dy.astype(np.float64) * w)
    d = r[:, None] * (6 * U * g + n * (176 * U) * (g * n).mean(1, keepdims=True))
    d = d + (0 if ds is None else U * (np.abs(ds) + np.abs(rx)))
    assert np.all(np.abs(to_np(dx) - rx) <= d + HALF[dtype] * (np.abs(rx) + d))
    dwt = (rows + 516) * U * (np.abs(dy) * n).sum(0)
    assert np.all(np.abs(to_np(dw) - rw) <= dwt + U * np.abs(rw))
    # again: the same bits; without dw: the same dx; dx in dy's buffer
    dw2, dx2 = torch.empty_like(dw), torch.empty_like(dx)
    M.moe_rmsnorm_bwd(rows, h, dt, dev["dy"], dev["sum"], dev["rstd"], dev["w"], dev["dsum"], dx2, dw2, ws)
    assert torch.equal(dw, dw2) and torch.equal(dx, dx2)
    M.moe_rmsnorm_bwd(rows, h, dt, dev["dy"], dev["sum"], dev["rstd"], dev["w"], dev["dsum"], dev["dy"])
    assert torch.equal(dx, dev["dy"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,h,with_dsum", [(1, 128, True), (7, 7168, False), (700, 2048, True), (3000, 256, True),
                                              (3, 8320, True), (2, 65536, True), (400, 7168, True)])
def test_backward(rows, h, with_dsum, dtype):
    _check_bwd(lib(), rows, h, dtype, with_dsum, rows + h)


def test_gradient_against_differences():
    """fp32 forward runs at x + t d and x - t d: their loss differences agree with dx and dw."""
    M = lib()
    rows, h = 6, 256
    x, res, w = _inputs(rows, h, "f32", 8)
    rng = np.random.default_rng(9)
    dy = rng.standard_normal((rows, h)).astype(np.float32)
    f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731

    def fwd(x_, w_):
        s, y, r = f32(rows, h), f32(rows, h), f32(rows)
        M.moe_rmsnorm_fwd(rows, h, M.MOE_F32, to_dev(x_, "f32"), to_dev(res, "f32"), to_dev(w_, "f32"), EPS, s, y,
                          rstd=r)
        return s, y, r

    s, _, r = fwd(x, w)
    dx, dw = f32(rows, h), f32(h)
    ws = torch.empty(M.moe_rmsnorm_bwd_workspace_size(rows, h), dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm_bwd(rows, h, M.MOE_F32, to_dev(dy, "f32"), s, r, to_dev(w, "f32"), None, dx, dw, ws)
    loss = lambda x_, w_: float((to_np(fwd(x_, w_)[1]).astype(np.float64) * dy).sum())  # noqa: E731
    t = 2.0 ** -6
    for k in range(3):
        d, e = rng.standard_normal((rows, h)).astype(np.float32), rng.standard_normal(h).astype(np.float32)
        # the third-order term is below t^2 |d|^3 r^3 |dy| a value, and the y's are within 2^-17 of theirs
        noise = 2 * 2.0 ** -17 * float(np.abs(to_np(fwd(x, w)[1]) * dy).sum()) / (2 * t)
        got = (loss(x + t * d, w) - loss(x - t * d, w)) / (2 * t)
        assert abs(got - float((to_np(dx).astype(np.float64) * d).sum())) <= noise + t * t * np.abs(d ** 3 * dy).sum()
        got = (loss(x, w + t * e) - loss(x, w - t * e)) / (2 * t)
        assert abs(got - float((to_np(dw).astype(np.float64) * e).sum())) <= noise


def test_no_rows():
    M = lib()
    dw = torch.full((256,), 3.0, device="cuda")
    z = torch.empty(0, 256, device="cuda")
    M.moe_rmsnorm_fwd(0, 256, M.MOE_F32, z, None, dw, EPS, y=z)
    M.moe_rmsnorm_bwd(0, 256, M.MOE_F32, None, None, None, None, None, None, dw)
    assert torch.all(dw == 0)


def test_side_stream_and_replays():
    """Forward and backward captured together on a side stream, replayed on new inputs."""
    M = lib()
    rows, h = 300, 1024
    w = to_dev(_inputs(1, h, "bf16", 1)[2], "f32")
    bf = lambda: torch.zeros(rows, h, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, res, dy, s, y, dx = (bf() for _ in range(6))
    q, sf = torch.zeros(rows, h, dtype=torch.uint8, device="cuda"), torch.zeros(rows, h // 128, device="cuda")
    r, dw = torch.zeros(rows, device="cuda"), torch.zeros(h, device="cuda")
    ws = torch.empty(M.moe_rmsnorm_bwd_workspace_size(rows, h), dtype=torch.uint8, device="cuda")

    def step():
        M.moe_rmsnorm_fwd(rows, h, M.MOE_BF16, x, res, w, EPS, s, y, q, sf, r)
        M.moe_rmsnorm_bwd(rows, h, M.MOE_BF16, dy, s, r, w, y, dx, dw, ws)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    outs = (s, y, q, sf, r, dx, dw)
    for seed in (11, 12):
        a, b, _ = _inputs(rows, h, "bf16", seed)
        x.copy_(to_dev(a, "bf16")), res.copy_(to_dev(b, "bf16")), dy.copy_(to_dev(a[::-1].copy(), "bf16"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        step()
        torch.cuda.synchronize()
        for t, u in zip(outs, got):
            assert torch.equal(t.view(torch.uint8), u.view(torch.uint8))
        check_fwd(a, b, to_np(w), "bf16", s, y, q, sf, r)
