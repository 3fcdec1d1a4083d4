"""GPU parity of MXFP4: moe_mxfp4_quantize / moe_mxfp4_dequantize bit-exact
against the oracle, and the grouped expert products.

Tolerances of the products: the operands' values are exact, so with K products
of magnitude |a_k b_k| summed in fp32, each of the K additions off by at most one
unit of the last place of a partial sum (2^-23, a truncating adder included),
|gpu - exact| <= K 2^-23 sum_k |a_k b_k|; a bf16 output adds half a step,
2^-8 |out|.  FC1 carries the bound of gate and up through p silu(g) u with
|silu'| <= 1.1, plus 2^-18 |a| for the fp32 evaluation."""

import numpy as np
import pytest
import torch

from gpu_util import lib, needs_gpu, to_dev, to_np
from oracle import mxfp4_oracle as X4
from oracle.mxfp8_oracle import silu

pytestmark = [pytest.mark.gpu, needs_gpu]

U = 2.0 ** -23


def bf16(a):
    return to_np(torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16))


def scale_index(rows, K, offsets=None, urows=None):
    """Byte of each (row, block) scale in the documented atoms; rows of no group: -1."""
    KB = K // 128
    r = np.arange(rows)
    if offsets is not None:
        offs = np.asarray(offsets, np.int64)
        inside = (r >= offs[0]) & (r < offs[-1])
        g = np.clip(np.searchsorted(offs, r, side="right") - 1, 0, len(offs) - 2)
        rt = np.concatenate([[0], np.cumsum((np.diff(offs) + 127) // 128)])
        lr = r - offs[g]
        tile = rt[g] + lr // 128
    else:
        inside = np.ones(rows, bool)
        lr = r % urows
        tile = (r // urows) * ((urows + 127) // 128) + lr // 128
    i = lr % 128
    base = (tile[:, None] * KB + np.arange(KB)) * 512 + (16 * (i % 32) + 4 * (i // 32))[:, None]
    idx = (base[:, :, None] + np.arange(4)).reshape(rows, KB * 4)
    idx[~inside] = -1
    return idx


def scales_of(sf, idx):
    s = sf.cpu().numpy()
    return np.where(idx >= 0, s[np.maximum(idx, 0)], 0).astype(np.uint8)


def quantize_dev(M, x, groups, offsets=None):
    rows, K = x.shape
    q = torch.full((rows, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(M.moe_mxfp8_scale_bytes(rows, K, groups), dtype=torch.uint8, device="cuda")
    od = None if offsets is None else torch.from_numpy(np.asarray(offsets, np.int32)).cuda()
    M.moe_mxfp4_quantize(rows, K, groups, od, to_dev(x, "bf16"), q, sf)
    return q, sf


def hard_rows(rng, rows, K):
    """A wide range, a zero block, subnormals, exact ties, non-finite values."""
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-40, 40, (rows, 1)))
    if rows > 5:
        x[1, :32] = 0.0
        x[2, 32:64] = rng.standard_normal(32) * 2.0 ** -130          # bf16 subnormals
        mids = (X4.LADDER[1:] + X4.LADDER[:-1]) / 2
        blk = np.concatenate([[6.0], rng.choice(mids, 31)]) * 2.0 ** 5
        x[3, :32] = blk * np.where(rng.random(32) < 0.5, -1, 1)
        x[4, 5], x[4, 70] = np.inf, np.nan
        x[5, :32] = 2.0 ** 127 * 1.5
    return bf16(x)


SHAPES = [
    (1000, 256, [0, 300, 300, 301, 900], 4),        # an empty and a one-row group, 100 rows outside
    (300, 7168, None, 3),                            # uniform groups of 100 rows
    (640, 2048, None, 5),                            # uniform groups of 128
    (777, 384, [0, 129, 256, 257, 777], 4),
    (50, 128, [7, 7, 40], 2),                        # rows before the first group
    (1, 128, [0, 1], 1),
]


@pytest.mark.parametrize("rows,K,offsets,groups", SHAPES)
def test_quantize_and_dequantize_bit_exact(rows, K, offsets, groups):
    M = lib()
    x = hard_rows(np.random.default_rng(rows + K), rows, K)
    q, sf = quantize_dev(M, x, groups, offsets)
    oq, os_ = X4.quantize(x)
    np.testing.assert_array_equal(q.cpu().numpy(), oq)
    idx = scale_index(rows, K, offsets, None if offsets is not None else rows // groups)
    ok = idx >= 0
    assert ok.any()
    np.testing.assert_array_equal(scales_of(sf, idx)[ok], os_[ok])
    out = torch.full((rows, K), -77.0, dtype=torch.bfloat16, device="cuda")
    od = None if offsets is None else torch.from_numpy(np.asarray(offsets, np.int32)).cuda()
    M.moe_mxfp4_dequantize(rows, K, groups, od, q, sf, out)
    want = X4.dequantize(oq, os_)
    want[~ok[:, 0]] = -77.0                          # rows of no group stay as they were
    np.testing.assert_array_equal(to_np(out).astype(np.float64), want)


def test_dequantize_every_code_and_scale():
    M = lib()
    rows = 256                                        # scale code = row, 16 codes twice a block
    codes = np.tile(np.arange(16, dtype=np.uint8), 8)
    q = torch.from_numpy(np.tile(codes[0::2] | (codes[1::2] << 4), (rows, 1))).cuda()
    idx = scale_index(rows, 128, None, rows)
    sf = np.zeros(M.moe_mxfp8_scale_bytes(rows, 128, 1), np.uint8)
    sf[idx] = np.arange(rows)[:, None]
    out = torch.empty(rows, 128, dtype=torch.bfloat16, device="cuda")
    M.moe_mxfp4_dequantize(rows, 128, 1, None, q, torch.from_numpy(sf).cuda(), out)
    want = X4.dequantize(q.cpu().numpy(), np.tile(np.arange(rows)[:, None], (1, 4)))
    want = torch.from_numpy(want).to(torch.bfloat16).float().numpy()   # 6 2^126 and up: infinite
    np.testing.assert_array_equal(to_np(out), want)


def _case(seed, T, K, E, h, F, skew=False, empty=()):
    rng = np.random.default_rng(seed)
    P = T * K
    w = rng.dirichlet(np.full(E, 0.3)) if skew else np.ones(E)
    for e in empty:
        w[e] = 0.0
    offsets = np.concatenate([[0], np.cumsum(rng.multinomial(P, w / w.sum()))]).astype(np.int64)
    return dict(T=T, K=K, E=E, h=h, F=F, P=P, offsets=offsets, x=bf16(rng.standard_normal((P, h))),
                w1=bf16(rng.standard_normal((E * 2 * F, h)) / np.sqrt(h)),
                w2=bf16(rng.standard_normal((E * h, F)) / np.sqrt(F)),
                p=rng.uniform(0.05, 1.0, P).astype(np.float32))


def _fc1_bound(A, offs, B, F, Kd, p):
    H = X4.grouped_gemm(A, offs, B, 2 * F)
    t = Kd * U * X4.grouped_gemm(np.abs(A), offs, np.abs(B), 2 * F)
    g, u, tg, tu = H[:, :F], H[:, F:], t[:, :F], t[:, F:]
    pp = p.astype(np.float64)[:, None]
    a = pp * silu(g) * u
    d = pp * (1.1 * tg * (np.abs(u) + tu) + (np.abs(silu(g)) + 1.1 * tg) * tu)
    return a, d + 2.0 ** -18 * np.abs(a) + 1e-30


CASES = [
    dict(seed=1, T=300, K=2, E=8, h=256, F=128),
    dict(seed=2, T=500, K=4, E=16, h=384, F=256, skew=True, empty=(3, 7)),   # half a last stage
    dict(seed=3, T=100, K=8, E=64, h=512, F=128, skew=True),                 # experts below one tile
    dict(seed=4, T=2048, K=1, E=2, h=1024, F=384),                           # several tiles an expert
    dict(seed=5, T=1, K=1, E=3, h=128, F=128),                               # one row, half a stage
    dict(seed=6, T=1024, K=2, E=4, h=2048, F=640),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: f"T{c['T']}_E{c['E']}_h{c['h']}_F{c['F']}")
def test_fc1_fc2_match_oracle(c):
    M = lib()
    c = _case(**c)
    P, E, h, F, offs = c["P"], c["E"], c["h"], c["F"], c["offsets"]
    cfg = M.make_config(c["T"], h, E, c["K"], F)
    od = torch.from_numpy(offs.astype(np.int32)).cuda()
    xq, xsf = quantize_dev(M, c["x"], E, offs)
    w1q, w1sf = quantize_dev(M, c["w1"], E)
    w2q, w2sf = quantize_dev(M, c["w2"], E)
    a = torch.full((P, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    aq = torch.empty(P, F // 2, dtype=torch.uint8, device="cuda")
    asf = torch.zeros(M.moe_mxfp8_scale_bytes(P, F, E), dtype=torch.uint8, device="cuda")
    pd = torch.from_numpy(c["p"]).cuda()
    M.moe_expert_fc1_mxfp4(cfg, xq, xsf, od, pd, w1q, w1sf, a, aq, asf)
    y = torch.full((P, h), float("nan"), dtype=torch.bfloat16, device="cuda")
    M.moe_expert_fc2_mxfp4(cfg, aq, asf, od, w2q, w2sf, y)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    A, B = X4.dequantize(*X4.quantize(c["x"])), X4.dequantize(*X4.quantize(c["w1"]))
    a_ref, d = _fc1_bound(A, offs, B, F, h, c["p"])
    ag = to_np(a).astype(np.float64)
    tol = d + 2.0 ** -8 * (np.abs(a_ref) + d)
    assert np.all(np.abs(ag - a_ref) <= tol), float((np.abs(ag - a_ref) / tol).max())
    # the 4-bit a: half a step of its block's scale (1/4 relative, scale / 4
    # below the normal range), magnitudes beyond 6 scales saturated
    ac, as_ = aq.cpu().numpy(), scales_of(asf, scale_index(P, F, offs))
    deq, sc = X4.dequantize(ac, as_), np.repeat(np.exp2(as_.astype(float) - 127), 32, axis=1)
    mag = np.abs(a_ref) + d
    tol = d + np.maximum(mag, sc) * 0.25 + np.maximum(mag - 6 * sc, 0)
    assert np.all(np.abs(deq - a_ref) <= tol)
    amax, dmax = (v.reshape(P, F // 32, 32).max(2) for v in (np.abs(a_ref), d))
    lo = np.floor(np.log2(np.maximum(amax - dmax, 2.0 ** -125))) + 125
    hi = np.floor(np.log2(amax + dmax)) + 125
    assert np.all((as_ >= lo) & (as_ <= hi)) and np.mean(lo == hi) > 0.8
    # FC2 on the GPU's own 4-bit a
    B2 = X4.dequantize(*X4.quantize(c["w2"]))
    y_ref = X4.grouped_gemm(deq, offs, B2, h)
    S = X4.grouped_gemm(np.abs(deq), offs, np.abs(B2), h)
    tol = F * U * S + 2.0 ** -8 * np.abs(y_ref) + 1e-30
    yg = to_np(y).astype(np.float64)
    assert np.all(np.abs(yg - y_ref) <= tol), float((np.abs(yg - y_ref) / tol).max())


def test_outputs_alone_null_prob_and_reruns_bitwise():
    M = lib()
    c = _case(seed=7, T=400, K=2, E=8, h=256, F=256, skew=True)
    P, E, h, F, offs = c["P"], c["E"], c["h"], c["F"], c["offsets"]
    cfg = M.make_config(c["T"], h, E, c["K"], F)
    od = torch.from_numpy(offs.astype(np.int32)).cuda()
    xq, xsf = quantize_dev(M, c["x"], E, offs)
    w1q, w1sf = quantize_dev(M, c["w1"], E)
    outs = []
    for want_a, want_q in ((True, False), (False, True), (True, True)):
        a = torch.empty(P, F, dtype=torch.bfloat16, device="cuda") if want_a else None
        aq = torch.empty(P, F // 2, dtype=torch.uint8, device="cuda") if want_q else None
        asf = torch.zeros(M.moe_mxfp8_scale_bytes(P, F, E), dtype=torch.uint8,
                          device="cuda") if want_q else None
        M.moe_expert_fc1_mxfp4(cfg, xq, xsf, od, None, w1q, w1sf, a, aq, asf)
        outs.append((a, aq, asf))
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    assert torch.equal(outs[0][0], outs[2][0])
    idx = scale_index(P, F, offs)
    assert torch.equal(outs[1][1], outs[2][1])
    assert np.array_equal(scales_of(outs[1][2], idx), scales_of(outs[2][2], idx))
    A, B = X4.dequantize(*X4.quantize(c["x"])), X4.dequantize(*X4.quantize(c["w1"]))
    a_ref, d = _fc1_bound(A, offs, B, F, h, np.ones(P, np.float32))
    ag = to_np(outs[0][0]).astype(np.float64)
    assert np.all(np.abs(ag - a_ref) <= d + 2.0 ** -8 * (np.abs(a_ref) + d))


def test_non_finite_rows_stay_in_their_rows():
    """A row with an infinity or a NaN gives NaN in its own outputs only."""
    M = lib()
    c = _case(seed=8, T=200, K=1, E=4, h=256, F=128)
    P, E, h, F, offs = c["P"], c["E"], c["h"], c["F"], c["offsets"]
    cfg = M.make_config(c["T"], h, E, 1, F)
    od = torch.from_numpy(offs.astype(np.int32)).cuda()
    w1q, w1sf = quantize_dev(M, c["w1"], E)
    outs = []
    for x in (c["x"], c["x"].copy()):
        if outs:
            x[17, 3], x[150, 200] = np.inf, np.nan
        xq, xsf = quantize_dev(M, x, E, offs)
        a = torch.zeros(P, F, dtype=torch.bfloat16, device="cuda")
        M.moe_expert_fc1_mxfp4(cfg, xq, xsf, od, None, w1q, w1sf, a, None, None)
        outs.append(to_np(a))
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    rest = np.setdiff1d(np.arange(P), [17, 150])
    np.testing.assert_array_equal(outs[0][rest], outs[1][rest])
    assert np.isnan(outs[1][[17, 150]]).all()


def test_two_streams_and_graph_replay():
    """Calls on a side stream, and a captured quantise + FC1 replayed on new inputs."""
    M = lib()
    c = _case(seed=9, T=150, K=2, E=4, h=256, F=128)
    P, E, h, F, offs = c["P"], c["E"], c["h"], c["F"], c["offsets"]
    cfg = M.make_config(c["T"], h, E, c["K"], F)
    od = torch.from_numpy(offs.astype(np.int32)).cuda()
    w1q, w1sf = quantize_dev(M, c["w1"], E)
    x = to_dev(c["x"], "bf16")
    xq = torch.empty(P, h // 2, dtype=torch.uint8, device="cuda")
    xsf = torch.zeros(M.moe_mxfp8_scale_bytes(P, h, E), dtype=torch.uint8, device="cuda")
    a = torch.empty(P, F, dtype=torch.bfloat16, device="cuda")

    def step():
        M.moe_mxfp4_quantize(P, h, E, od, x, xq, xsf)
        M.moe_expert_fc1_mxfp4(cfg, xq, xsf, od, None, w1q, w1sf, a, None, None)

    step()
    torch.cuda.synchronize()
    want = a.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a.zero_()
        step()
    s.synchronize()
    assert torch.equal(a, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.copy_(-x)
    g.replay()
    torch.cuda.synchronize()
    got = a.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(a, got) and not torch.equal(a, want)
    assert M.moe_get_error() == M.MOE_OK


def test_nothing_is_written_outside_the_buffers():
    """Codes, scales, values and product outputs between guard bytes."""
    M = lib()
    for rows, K, offsets, groups in SHAPES:
        x = to_dev(hard_rows(np.random.default_rng(rows), rows, K), "bf16")
        nsf, G = M.moe_mxfp8_scale_bytes(rows, K, groups), 4096
        q = torch.full((rows * K // 2 + 2 * G,), 0x77, dtype=torch.uint8, device="cuda")
        sf = torch.full((nsf + 2 * G,), 0x77, dtype=torch.uint8, device="cuda")
        out = torch.full((rows * K + 2 * G,), 5.0, dtype=torch.bfloat16, device="cuda")
        od = None if offsets is None else torch.from_numpy(np.asarray(offsets, np.int32)).cuda()
        M.moe_mxfp4_quantize(rows, K, groups, od, x, q[G:-G], sf[G:-G])
        M.moe_mxfp4_dequantize(rows, K, groups, od, q[G:-G], sf[G:-G], out[G:-G])
        torch.cuda.synchronize()
        for b, v in ((q, 0x77), (sf, 0x77), (out, 5.0)):
            assert (b[:G] == v).all() and (b[-G:] == v).all()
    c = _case(seed=11, T=131, K=2, E=5, h=384, F=128, skew=True)
    P, E, h, F, offs = c["P"], c["E"], c["h"], c["F"], c["offsets"]
    cfg = M.make_config(c["T"], h, E, c["K"], F)
    od = torch.from_numpy(offs.astype(np.int32)).cuda()
    xq, xsf = quantize_dev(M, c["x"], E, offs)
    w1q, w1sf = quantize_dev(M, c["w1"], E)
    w2q, w2sf = quantize_dev(M, c["w2"], E)
    u8 = dict(dtype=torch.uint8, device="cuda")
    nsf = M.moe_mxfp8_scale_bytes(P, F, E)
    for shift in (0, 8):                # outputs on a 32-byte boundary, and 16 bytes off it
        a = torch.full((P * F + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
        y = torch.full((P * h + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
        aq, asf = torch.full((P * F // 2 + 64,), 0x77, **u8), torch.full((nsf + 64,), 0x77, **u8)
        av, yv = a[16 + shift:16 + shift + P * F], y[16 + shift:16 + shift + P * h]
        M.moe_expert_fc1_mxfp4(cfg, xq, xsf, od, None, w1q, w1sf, av, aq[32:-32], asf[32:-32])
        M.moe_expert_fc2_mxfp4(cfg, aq[32:-32], asf[32:-32], od, w2q, w2sf, yv)
        torch.cuda.synchronize()
        assert M.moe_get_error() == M.MOE_OK
        for b, v in ((aq, 0x77), (asf, 0x77)):
            assert (b[:32] == v).all() and (b[-32:] == v).all()
        for b, n in ((a, P * F), (y, P * h)):
            assert (b[:16 + shift] == 5).all() and (b[16 + shift + n:] == 5).all()
        if shift == 0:
            first = av.clone(), yv.clone()
        else:
            assert torch.equal(av, first[0]) and torch.equal(yv, first[1])


def test_descending_offsets_stay_in_bounds():
    """Offsets are the caller's promise; a broken one must not reach past the
    scale buffer (the kernel cuts boundaries to the rows and tiles to the room)."""
    M = lib()
    rows, K, G = 300, 256, 6
    off = torch.tensor([0, 300, 0, 300, -5, 300, 1 << 30], dtype=torch.int32, device="cuda")
    n = M.moe_mxfp8_scale_bytes(rows, K, G)
    x = torch.ones(rows, K, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.full((n + 8192,), 0x77, dtype=torch.uint8, device="cuda")
    out = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    M.moe_mxfp4_quantize(rows, K, G, off, x, q, sf[:n])
    M.moe_mxfp4_dequantize(rows, K, G, off, q, sf[:n], out)
    torch.cuda.synchronize()
    assert (sf[n:] == 0x77).all()


def test_injected_failure_enqueues_nothing():
    M = lib()
    x = torch.ones(16, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.full((16, 64), 0x77, dtype=torch.uint8, device="cuda")
    sf = torch.full((M.moe_mxfp8_scale_bytes(16, 128, 1),), 0x77, dtype=torch.uint8, device="cuda")
    assert M.moe_test_inject_cuda_failure(1) == 0
    with pytest.raises(M.MoeError):
        M.moe_mxfp4_quantize(16, 128, 1, None, x, q, sf)
    torch.cuda.synchronize()
    assert (q == 0x77).all() and (sf == 0x77).all()


def test_products_keep_broken_offsets_within_the_rows():
    """Offsets past the last row end there; descending ones reach past no tensor."""
    M = lib()
    c = _case(seed=12, T=140, K=1, E=5, h=256, F=128)
    P, E, h, F, offs = c["P"], c["E"], c["h"], c["F"], c["offsets"]
    cfg = M.make_config(c["T"], h, E, c["K"], F)
    xq, xsf = quantize_dev(M, c["x"], E, offs)
    w1q, w1sf = quantize_dev(M, c["w1"], E)
    w2q, w2sf = quantize_dev(M, c["w2"], E)
    nsf, G = M.moe_mxfp8_scale_bytes(P, F, E), 4096
    past = offs.astype(np.int64).copy()
    past[-1] = 1 << 30
    outs = []
    for o in (offs, past, np.array([P, 0, P, -9, 1 << 30, 3]), np.array([-5, 1 << 30, 0, 17, 2, 1])):
        od = torch.from_numpy(o.astype(np.int32)).cuda()
        a = torch.full((P * F + 2 * G,), 5.0, dtype=torch.bfloat16, device="cuda")
        y = torch.full((P * h + 2 * G,), 5.0, dtype=torch.bfloat16, device="cuda")
        aq = torch.full((P * F // 2 + 2 * G,), 0x77, dtype=torch.uint8, device="cuda")
        asf = torch.full((nsf + 2 * G,), 0x77, dtype=torch.uint8, device="cuda")
        M.moe_expert_fc1_mxfp4(cfg, xq, xsf, od, None, w1q, w1sf, a[G:-G], aq[G:-G], asf[G:-G])
        M.moe_expert_fc2_mxfp4(cfg, aq[G:-G], asf[G:-G], od, w2q, w2sf, y[G:-G])
        torch.cuda.synchronize()
        assert M.moe_get_error() == M.MOE_OK
        for b, v in ((a, 5.0), (y, 5.0), (aq, 0x77), (asf, 0x77)):
            assert (b[:G] == v).all() and (b[-G:] == v).all()
        outs.append((a.clone(), y.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_fc1_quantised_output_of_non_finite_blocks():
    """A block of a with a NaN: the NaN scale and zero codes, as the quantiser writes it."""
    M = lib()
    c = _case(seed=13, T=40, K=1, E=2, h=128, F=256)
    P, E, h, F, offs = c["P"], c["E"], c["h"], c["F"], c["offsets"]
    cfg = M.make_config(c["T"], h, E, c["K"], F)
    x = c["x"].copy()
    x[3, 7] = np.nan
    xq, xsf = quantize_dev(M, x, E, offs)
    w1q, w1sf = quantize_dev(M, c["w1"], E)
    od = torch.from_numpy(offs.astype(np.int32)).cuda()
    aq = torch.full((P, F // 2), 0x77, dtype=torch.uint8, device="cuda")
    asf = torch.zeros(M.moe_mxfp8_scale_bytes(P, F, E), dtype=torch.uint8, device="cuda")
    M.moe_expert_fc1_mxfp4(cfg, xq, xsf, od, None, w1q, w1sf, None, aq, asf)
    torch.cuda.synchronize()
    assert M.moe_get_error() == M.MOE_OK
    sc = scales_of(asf, scale_index(P, F, offs))
    assert (sc[3] == 255).all() and (aq[3] == 0).all()
    rest = np.setdiff1d(np.arange(P), [3])
    assert (sc[rest] != 255).all()
