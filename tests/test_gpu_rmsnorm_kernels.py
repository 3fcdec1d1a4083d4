"""The RMS norm's kernels one by one against the float64 oracle: the forward for rows of
1024 to 8192 columns of larger batches, each form of the gradient's ring (groups of 1 to 16
warps, one or several rows a stage, w inside and outside shared memory), the gradient of
longer rows, and the gradient in place with dw.

Tolerances (U = 2^-24, half a step of fp32).  The forward's are test_gpu_rmsnorm's: its sums
pass at most 64 + 5 + 32 additions one after the other.  A dot product of the gradient adds
8 ceil(h / 2048) products a thread where a block of 256 has a row (up to 512 rows, not in
place), else at most 64, then 5 times in a warp and once for each of at most 32 warps; each
product has two roundings before it and the mean two after.  So the mean of g n is within
(max(8 ceil(h / 2048), 64) + 41) U of the mean of |g n|; dx carries that times r |n|, 6
roundings of g, and the residual's addition.  dw adds one product a row, at most rows + 512
times."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu, to_dev, to_np
from oracle import fp8_oracle as X
from test_gpu_rmsnorm import DT, EPS, HALF, U, _inputs, check_fwd, rounded

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,h", [(400, 2048), (401, 4096), (400, 7168), (333, 8192), (700, 1152)])
def test_forward_of_larger_batches(rows, h, dtype):
    M = lib()
    x, res, w = _inputs(rows, h, dtype, rows + h)
    xd, rd, wd = to_dev(x, dtype), to_dev(res, dtype), to_dev(w, "f32")
    e = lambda *s, dt=DT[dtype]: torch.full(s, 77, dtype=dt, device="cuda")  # noqa: E731
    o = dict(sum=e(rows, h), y=e(rows, h), q=e(rows, h, dt=torch.uint8), sf=e(rows, h // 128, dt=torch.float32),
             rstd=e(rows, dt=torch.float32))
    dt = M.MOE_BF16 if dtype == "bf16" else M.MOE_F32
    M.moe_rmsnorm_fwd(rows, h, dt, xd, rd, wd, EPS, **o)
    check_fwd(x, res, w, dtype, **o)
    y2, q2, sf2 = e(rows, h), e(rows, h, dt=torch.uint8), e(rows, h // 128, dt=torch.float32)
    M.moe_rmsnorm_fwd(rows, h, dt, xd, None, wd, EPS, y=y2, q=q2, sf=sf2)
    check_fwd(x, None, w, dtype, y=y2, q=q2, sf=sf2)
    # the sum in the residual's buffer, y in x's
    M.moe_rmsnorm_fwd(rows, h, dt, xd, rd, wd, EPS, rd, xd)
    assert torch.equal(rd, o["sum"]) and torch.equal(xd, o["y"])


@pytest.mark.parametrize("dtype,rows,h", [("bf16", 400, 2056), ("bf16", 300, 7000), ("f32", 400, 2052), ("f32", 300, 7004),
                                          ("f32", 200, 1028)])
def test_forward_of_odd_widths_in_larger_batches(dtype, rows, h):
    M = lib()
    x, res, w = _inputs(rows, h, dtype, h)
    pad = torch.full((2, rows * h + 64), 55.0, dtype=DT[dtype], device="cuda")
    s, y = (p[:rows * h].view(rows, h) for p in pad)
    rstd = torch.empty(rows, device="cuda")
    M.moe_rmsnorm_fwd(rows, h, M.MOE_BF16 if dtype == "bf16" else M.MOE_F32, to_dev(x, dtype), to_dev(res, dtype),
                      to_dev(w, "f32"), EPS, s, y, rstd=rstd)
    check_fwd(x, res, w, dtype, sum=s, y=y, rstd=rstd)
    assert torch.all(pad[:, rows * h:] == 55.0)


class Case:
    """A gradient's inputs, what it should be and how far it may be from that."""

    def __init__(self, M, rows, h, dtype, with_dsum):
        rng = np.random.default_rng(rows + h)
        self.M, self.rows, self.h, self.dtype = M, rows, h, dtype
        self.dt = M.MOE_BF16 if dtype == "bf16" else M.MOE_F32
        v = rounded(2 * rng.standard_normal((rows, h), np.float32), dtype)
        dy = rounded(rng.standard_normal((rows, h), np.float32), dtype)
        ds = rounded(rng.standard_normal((rows, h), np.float32), dtype) if with_dsum else None
        w = (1 + 0.1 * rng.standard_normal(h)).astype(np.float32)
        r = (1 / np.sqrt((v.astype(np.float64) ** 2).mean(1) + EPS)).astype(np.float32)
        self.dev = dict(dy=to_dev(dy, dtype), sum=to_dev(v, dtype), rstd=to_dev(r, "f32"), w=to_dev(w, "f32"),
                        dsum=None if ds is None else to_dev(ds, dtype))
        self.ws = torch.full((M.moe_rmsnorm_bwd_workspace_size(rows, h),), 0xEE, dtype=torch.uint8, device="cuda")
        self.rx, self.rw = X.rmsnorm_bwd(dy, v, r, w, ds)
        n = np.abs(v.astype(np.float64)) * r[:, None]
        g = np.abs(dy.astype(np.float64) * w)
        m = (max(8 * -(-h // 2048), 64) + 41) * U * (g * n).mean(1, keepdims=True)
        d = r[:, None] * (6 * U * g + n * m)
        if ds is not None:
            d += U * (np.abs(ds) + np.abs(self.rx))
        self.tx = d + HALF[dtype] * (np.abs(self.rx) + d)
        self.tw = (rows + 516) * U * (np.abs(dy) * n).sum(0) + U * np.abs(self.rw)

    def run(self, dx=None, dw=True, **over):
        dx = torch.full((self.rows, self.h), 77.0, dtype=DT[self.dtype], device="cuda") if dx is None else dx
        dw = torch.full((self.h,), 77.0, device="cuda") if dw else None
        a = {**self.dev, **over}
        self.M.moe_rmsnorm_bwd(self.rows, self.h, self.dt, a["dy"], a["sum"], a["rstd"], a["w"], a["dsum"], dx, dw,
                               self.ws if dw is not None else None)
        return dx, dw

    def check(self, dx, dw):
        assert self.M.moe_get_error() == self.M.MOE_OK
        assert np.all(np.abs(to_np(dx) - self.rx) <= self.tx)
        if dw is not None:
            assert np.all(np.abs(to_np(dw) - self.rw) <= self.tw)

    def in_place(self):
        """dx in dy's, sum's and dsum's own buffer, with dw and without."""
        for name in ("dy", "sum", "dsum"):
            if self.dev[name] is None:
                continue
            for with_dw in (True, False):
                buf = self.dev[name].clone()
                dx, dw = self.run(buf, with_dw, **{name: buf})
                self.check(dx, dw)


GRADIENTS = [
    ("bf16", 2001, 7168, True), ("bf16", 700, 7168, False), ("f32", 700, 7168, True), ("f32", 2001, 7168, False),
    ("f32", 1300, 8192, True), ("f32", 600, 7904, True),                # w outside shared memory
    ("bf16", 600, 8192, True), ("bf16", 1300, 8192, False),
    ("bf16", 520, 5000, True), ("f32", 2500, 4100, True), ("f32", 513, 1028, True),
    ("bf16", 3000, 1032, False), ("bf16", 900, 696, False), ("f32", 700, 1004, False), ("f32", 5000, 1024, True),
    ("bf16", 2000, 200, False), ("f32", 4000, 36, True), ("f32", 6001, 512, False), ("bf16", 20011, 8, True),
    ("bf16", 9001, 1000, True),
    ("bf16", 600, 8320, True), ("f32", 600, 8196, False),               # longer rows
    ("bf16", 520, 33000, True), ("f32", 520, 33000, False), ("bf16", 516, 65536, False),
]


@pytest.mark.parametrize("dtype,rows,h,with_dsum", GRADIENTS)
def test_gradient(dtype, rows, h, with_dsum):
    c = Case(lib(), rows, h, dtype, with_dsum)
    dx, dw = c.run()
    c.check(dx, dw)
    dx2, dw2 = c.run()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)               # again: the same bits
    assert torch.equal(c.run(dw=False)[0], dx)
    # dx behind a buffer's start: nothing outside its rows
    pad = torch.full((rows * h + 128,), 55.0, dtype=DT[dtype], device="cuda")
    c.run(pad[64:64 + rows * h].view(rows, h))
    assert torch.equal(pad[64:64 + rows * h].view(rows, h), dx)
    assert torch.all(pad[:64] == 55.0) and torch.all(pad[64 + rows * h:] == 55.0)


@pytest.mark.parametrize("dtype,rows,h,with_dsum", [
    ("bf16", 1, 128, True), ("f32", 1, 4, True), ("bf16", 5, 7168, True), ("f32", 300, 2048, True), ("bf16", 512, 520, False),
    ("bf16", 2, 65536, True), ("f32", 3, 8196, True), ("bf16", 513, 1024, True), ("f32", 513, 8192, True),
    ("bf16", 2001, 4096, True), ("f32", 3000, 68, True), ("bf16", 600, 8320, True)])
def test_gradient_in_place(dtype, rows, h, with_dsum):
    c = Case(lib(), rows, h, dtype, with_dsum)
    c.check(*c.run())
    c.in_place()


def test_large_widths_of_few_rows():
    """A block of 256 threads a row: the longest sums one after the other."""
    for dtype, rows, h in (("f32", 2, 65536), ("bf16", 512, 9000), ("f32", 40, 30004)):
        c = Case(lib(), rows, h, dtype, True)
        c.check(*c.run())
