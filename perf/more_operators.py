"""Timed cases of the FP8 layer path: RMS norm with the residual's addition and
an 8-bit output (and its gradient), quantisation in blocks of 128, the grouped
expert products on FP8 operands with a scale for each block of 128, and rows
sorted by expert in 8 bits with the gradient of the weighted way back.

Every case gives the operator's plain form (elementary torch operations, sums
in 32 bits) and, with ``own`` set, the framework's call on the same inputs.
Inputs are made from the seed alone: activations and gradients N(0, 1), expert
weights N(0, 1/fan-in), norm weights near 1, skewed routing with each token's
experts distinct.  8-bit tensors are E4M3 codes (uint8) with one fp32 scale for
each 128 columns of a row (activations) or each 128 x 128 block (weights).
"""

import math

import numpy as np
import torch

own = False

BLOCK, TOP = 128, 448.0
EPS = 1e-6


# ---- cases ------------------------------------------------------------------------
def _norm(name, rows, h, dtype="bf16", res=True, y=True, q=True):
    return {"name": name, "op": "norm", "rows": rows, "h": h, "dtype": dtype, "res": res, "y": y, "q": q}


def _norm_bwd(name, rows, h, dtype="bf16", res=True):
    return {"name": name, "op": "norm_bwd", "rows": rows, "h": h, "dtype": dtype, "res": res}


def _quant(name, rows, cols):
    return {"name": name, "op": "quant", "rows": rows, "cols": cols}


def _quant_w(name, groups, rows, cols, both):
    return {"name": name, "op": "quant_w", "groups": groups, "rows": rows, "cols": cols, "both": both}


def _product(name, fc, T, h, E, K, F, q=False):
    return {"name": name, "op": "product", "fc": fc, "T": T, "h": h, "E": E, "K": K, "F": F, "q": q}


def _sort(name, T, h, E, K):
    return {"name": name, "op": "sort", "T": T, "h": h, "E": E, "K": K}


def _sort_bwd(name, T, h, E, K, dtype="bf16"):
    return {"name": name, "op": "sort_bwd", "T": T, "h": h, "E": E, "K": K, "dtype": dtype}


def listed():
    return [
        # the norm before the layer in one decoding step of seven sequences: latency
        _norm("norm_7x7168", 7, 7168),
        # a prefill batch: the residual stream, the router's bf16 rows and the experts' 8-bit ones
        _norm("norm_8192x4096", 8192, 4096),
        # a training batch's gradient, the residual stream's own among its inputs
        _norm_bwd("norm_bwd_4096x7168", 4096, 7168),
        # activations (or their gradients) that no norm quantises; an odd number of rows
        _quant("quant_1021x2048", 1021, 2048),
        # after an optimiser step: the first projections of 8 experts and their transposes
        _quant_w("quant_weights", 8, 28672, 4096, True),
        # a training or prefill batch over 8 experts, compute bound
        _product("fc1_T8192_E8", 1, 8192, 4096, 8, 2, 14336),
        # a chunk of a fine-grained layer: ragged, about 128 rows an expert
        _product("fc2_T512_E32", 2, 512, 7168, 32, 8, 2048),
        # a small decoding batch over many experts, the hidden values kept in 8 bits
        _product("fc1_T13_E64", 1, 13, 2048, 64, 8, 1024, q=True),
        # one sequence decoding: 8 of 256 experts, a row each
        _product("fc2_T1_E256", 2, 1, 7168, 256, 8, 2048),
        # rows of a large batch to their experts
        _sort("sort_16384x4096", 16384, 4096, 128, 8),
        # rows of a small, odd batch
        _sort("sort_333x2048", 333, 2048, 64, 8),
        # the gradient of the weighted way back
        _sort_bwd("sort_bwd_4096x7168", 4096, 7168, 256, 8),
    ]


def _log(rng, lo, hi, step):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def _experts(rng):
    E = rng.choice([4, 8, 32, 64, 128, 256])
    return E, rng.choice([k for k in (1, 2, 6, 8) if k <= E])


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quant", "quant_w", "product", "product", "sort", "sort_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        h = _log(rng, 128, 8192, 128)
        if op == "norm_bwd" or rng.random() < 0.2:  # without 8-bit rows, 16-byte rows are enough
            q, h = False, max(8, h - 8 * rng.randrange(0, 16))
        else:
            q = True
        rows = _log(rng, 1, max(2, min(16384, 32_000_000 // h)), 1)
        res = rng.random() < 0.7
        if op == "norm_bwd":
            c = _norm_bwd("", rows, h, dtype, res)
        else:
            c = _norm("", rows, h, dtype, res, not q or rng.random() < 0.6, q)
    elif op == "quant":
        cols = _log(rng, 128, 14336, 128)
        c = _quant("", _log(rng, 1, max(2, min(65536, 200_000_000 // cols)), 1), cols)
    elif op == "quant_w":
        cols, rows = _log(rng, 128, 14336, 128), _log(rng, 128, 14336, 128)
        c = _quant_w("", min(rng.choice([1, 3, 8, 64]), max(1, 500_000_000 // (rows * cols))), rows, cols,
                     rng.random() < 0.5)
    elif op == "product":
        E, K = _experts(rng)
        h = _log(rng, 512, 7168, 128)
        F = _log(rng, 256, 14336, 128)
        F = min(F, max(256, 1_500_000_000 // (E * h) // 128 * 128))
        T = _log(rng, 1, 8192, 1)
        T = max(1, min(T, int(1.5e12 // (4 * K * h * F))))
        fc = rng.choice([1, 2])
        c = _product("", fc, T, h, E, K, F, fc == 1 and rng.random() < 0.5)
    else:
        E, K = _experts(rng)
        h = _log(rng, 256, 7168, 128)
        T = _log(rng, 1, max(2, min(16384, 200_000_000 // (h * K))), 1)
        c = _sort("", T, h, E, K) if op == "sort" else _sort_bwd("", T, h, E, K, dtype)
    return {k: v for k, v in c.items() if k != "name"}


# ---- inputs -----------------------------------------------------------------------
def _gen(seed, tag):
    return torch.Generator(device="cuda").manual_seed(1_000_003 * int(seed) + tag)


def _normal(shape, std, seed, tag, dtype=torch.bfloat16):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, std, generator=_gen(seed, tag))


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _routing(T, E, K, seed):
    """Each token's K experts, distinct, by a skewed preference: [T, K]."""
    r = np.random.default_rng(int(seed))
    liked = np.log(r.dirichlet(np.full(E, 1.0)) + 1e-9)
    key = liked + r.gumbel(size=(T, E))
    return np.argsort(-key, axis=1)[:, :K].astype(np.int32)


def _codes(v, amax):
    """E4M3 codes of v 448 / amax, to nearest even, for block maxima that broadcast.
    The product is exact for 16-bit values, so that one division rounds and what
    lies on a border between two codes is seen as such."""
    return (v * TOP / amax).clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)


def _amax(b, *dims):
    for d in dims:
        b = b.abs().amax(d)
    return b.clamp(min=TOP * 2.0 ** -125)


def _quantize(v):
    """32-bit rows -> codes [rows, cols], scales [rows, cols / 128]."""
    b = v.view(v.shape[0], -1, BLOCK)
    a = _amax(b, 2)
    return _codes(b, a.unsqueeze(2)).view(v.shape), a / TOP


def _quantize_blocks(v):
    """32-bit [rows, cols] -> codes, scales [rows / 128, cols / 128]."""
    b = v.view(v.shape[0] // BLOCK, BLOCK, v.shape[1] // BLOCK, BLOCK)
    a = _amax(b, 3, 1)
    return _codes(b, a[:, None, :, None]).view(v.shape), a / TOP


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    c, op = case, case["op"]
    s = {"case": c}
    u8, f32, bf16, i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32
    if op in ("norm", "norm_bwd"):
        rows, h, dt = c["rows"], c["h"], _dtype(c)
        s["x"] = _normal((rows, h), 1.0, seed, 1, dt)
        s["res"] = _normal((rows, h), 2.0, seed, 2, dt) if c["res"] else None
        s["w"] = 1.0 + _normal((h,), 0.1, seed, 3, f32)
        if op == "norm":
            s["sum"] = _empty((rows, h), dt) if c["res"] else None
            s["y"] = _empty((rows, h), dt) if c["y"] else None
            s["q"] = _empty((rows, h), u8) if c["q"] else None
            s["sf"] = _empty((rows, h // BLOCK), f32) if c["q"] else None
            s["rstd"] = _empty((rows,), f32)
        else:  # what the forward left: the sum and 1 / rms of its rows
            s["dy"] = _normal((rows, h), 1.0, seed, 4, dt)
            s["sum"], s["dsum"] = s.pop("x"), s.pop("res")
            s["rstd"] = torch.rsqrt(s["sum"].float().square().mean(1) + EPS)
            s["dx"], s["dw"] = _empty((rows, h), dt), _empty((h,), f32)
    elif op == "quant":
        s["x"] = _normal((c["rows"], c["cols"]), 1.0, seed, 1)
        s["q"], s["sf"] = _empty((c["rows"], c["cols"]), u8), _empty((c["rows"], c["cols"] // BLOCK), f32)
    elif op == "quant_w":
        G, N, K = c["groups"], c["rows"], c["cols"]
        s["x"] = _normal((G, N, K), 1.0 / math.sqrt(K), seed, 1)
        s["q"], s["sf"] = _empty((G, N, K), u8), _empty((G, N // BLOCK, K // BLOCK), f32)
        s["q_t"] = _empty((G, K, N), u8) if c["both"] else None
        s["sf_t"] = _empty((G, K // BLOCK, N // BLOCK), f32) if c["both"] else None
    elif op == "product":
        T, h, E, K, F = c["T"], c["h"], c["E"], c["K"], c["F"]
        P = T * K
        kd, n = (h, 2 * F) if c["fc"] == 1 else (F, h)
        bounds = np.concatenate([[0], np.cumsum(np.bincount(_routing(T, E, K, seed).ravel(), minlength=E))])
        s["bounds"] = bounds.tolist()
        s["offsets"] = torch.from_numpy(bounds.astype(np.int32)).cuda()
        s["a_q"], s["a_sf"] = _quantize(_normal((P, kd), 1.0, seed, 1).float())
        s["w_q"], s["w_sf"] = _empty((E, n, kd), u8), _empty((E, n // BLOCK, kd // BLOCK), f32)
        g, w = _gen(seed, 2), _empty((n, kd), f32)
        for e in range(E):
            s["w_q"][e], s["w_sf"][e] = _quantize_blocks(w.normal_(0.0, 1.0 / math.sqrt(kd), generator=g))
        s["prob"] = torch.rand(P, device="cuda", generator=_gen(seed, 3)) if c["fc"] == 1 else None
        cols = F if c["fc"] == 1 else h
        s["out"] = None if c["q"] else _empty((P, cols), bf16)
        s["q"] = _empty((P, cols), u8) if c["q"] else None
        s["sf"] = _empty((P, cols // BLOCK), f32) if c["q"] else None
    else:
        T, h, E, K = c["T"], c["h"], c["E"], c["K"]
        P = T * K
        s["idx"] = torch.from_numpy(_routing(T, E, K, seed)).cuda()
        p = torch.rand((T, K), device="cuda", generator=_gen(seed, 3)) + 0.05
        s["prob"] = p / p.sum(1, keepdim=True)
        if op == "sort":
            s["x_q"], s["x_sf"] = _quantize(_normal((T, h), 1.0, seed, 1).float())
            s["q"], s["sf"] = _empty((P, h), u8), _empty((P, h // BLOCK), f32)
            s["counts"], s["offsets"] = _empty((E,), i32), _empty((E + 1,), i32)
            s["dst_row"], s["src_token"], s["perm_prob"] = _empty((T, K), i32), _empty((P,), i32), _empty((P,), f32)
        else:  # what the forward left: where each row went, and the experts' outputs
            s["dst_row"] = _order(s["idx"])[1].to(i32)
            s["dy"] = _normal((T, h), 1.0, seed, 1, _dtype(c))
            s["y_perm"] = _normal((P, h), 1.0, seed, 2, _dtype(c))
            s["dy_perm"], s["dprob"] = _empty((P, h), _dtype(c)), _empty((T, K), f32)
    return s


# ---- the framework's calls --------------------------------------------------------------
def _plan(M, s):
    """The config and workspace that a program makes once per layer and batch size."""
    c = s["case"]
    if c["op"] == "norm_bwd":
        cfg = None
        size = M.moe_rmsnorm_bwd_workspace_size(c["rows"], c["h"])
    else:
        cfg = M.make_config(c["T"], c["h"], c["E"], c["K"], c.get("F", c["h"]),
                            dtype=M.MOE_F32 if c.get("dtype") == "f32" else M.MOE_BF16)
        size = M.moe_workspace_size(cfg) if c["op"] == "sort" else 0
    s["plan"] = cfg, torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    return s["plan"]


def _run_own(s):
    from mixture_experts_layer_softmax_gb300 import moe as M
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        dt = M.MOE_BF16 if c["dtype"] == "bf16" else M.MOE_F32
        M.moe_rmsnorm_fwd(c["rows"], c["h"], dt, s["x"], s["res"], s["w"], EPS, s["sum"], s["y"], s["q"], s["sf"],
                          s["rstd"])
        return _named(s, "sum", "y", "q", "sf", "rstd")
    if op == "norm_bwd":
        dt = M.MOE_BF16 if c["dtype"] == "bf16" else M.MOE_F32
        _, ws = s.get("plan") or _plan(M, s)
        M.moe_rmsnorm_bwd(c["rows"], c["h"], dt, s["dy"], s["sum"], s["rstd"], s["w"], s["dsum"], s["dx"], s["dw"], ws)
        return _named(s, "dx", "dw")
    if op == "quant":
        M.moe_fp8_quantize(c["rows"], c["cols"], s["x"], s["q"], s["sf"])
        return _named(s, "q", "sf")
    if op == "quant_w":
        M.moe_fp8_quantize_weights(c["groups"], c["rows"], c["cols"], s["x"], s["q"], s["sf"], s["q_t"], s["sf_t"])
        return _named(s, "q", "sf", "q_t", "sf_t")
    cfg, ws = s.get("plan") or _plan(M, s)
    if op == "product":
        if c["fc"] == 1:
            M.moe_expert_fc1_fp8(cfg, s["a_q"], s["a_sf"], s["offsets"], s["prob"], s["w_q"], s["w_sf"], None,
                                 s["out"], s["q"], s["sf"])
        else:
            M.moe_expert_fc2_fp8(cfg, s["a_q"], s["a_sf"], s["offsets"], s["w_q"], s["w_sf"], s["out"])
        return _named(s, "out", "q", "sf")
    if op == "sort":
        M.moe_permute_fp8(cfg, s["x_q"], s["x_sf"], s["idx"], s["prob"], s["q"], s["sf"], s["counts"], s["offsets"],
                          s["dst_row"], s["src_token"], s["perm_prob"], ws)
        return _named(s, "q", "sf", "counts", "offsets", "dst_row", "src_token", "perm_prob")
    M.moe_unpermute_combine_bwd(cfg, s["dy"], s["y_perm"], s["dst_row"], s["prob"], s["dy_perm"], s["dprob"])
    return _named(s, "dy_perm", "dprob")


def _named(s, *names):
    """The outputs by name, 8-bit codes as the E4M3 numbers that they are."""
    out = {n: s[n] for n in names if s[n] is not None}
    return {n: v.view(torch.float8_e4m3fn) if v.dtype == torch.uint8 else v for n, v in out.items()}


# ---- the plain forms -----------------------------------------------------------------------
def _plain_norm(s):
    c, dt = s["case"], _dtype(s["case"])
    v = s["x"].float() + s["res"].float() if c["res"] else s["x"].float()
    rstd = 1.0 / torch.sqrt((v * v).mean(1) + EPS)
    y = v * rstd[:, None] * s["w"]
    out = {"rstd": rstd}
    if c["res"]:
        out["sum"] = v.to(dt)
    if c["y"]:
        out["y"] = y.to(dt)
    if c["q"]:
        out["q"], out["sf"] = _quantize(y)
    return out


def _plain_norm_bwd(s):
    n = s["sum"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"]
    dx = (g - n * (g * n).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["dy"].dtype), "dw": (dy * n).sum(0)}


def _values(q, sf):
    """The 32-bit values of codes [rows, cols] and scales [rows or rows / 128, cols / 128]."""
    s = sf.repeat_interleave(BLOCK, 1)
    if s.shape[0] != q.shape[0]:
        s = s.repeat_interleave(BLOCK, 0)
    return q.view(torch.float8_e4m3fn).float() * s


def _plain_product(s):
    c, F = s["case"], s["case"]["F"]
    x = _values(s["a_q"], s["a_sf"])
    out = torch.empty(x.shape[0], F if c["fc"] == 1 else c["h"], device="cuda")
    for e, (lo, hi) in enumerate(zip(s["bounds"][:-1], s["bounds"][1:])):
        if hi == lo:
            continue
        y = x[lo:hi] @ _values(s["w_q"][e], s["w_sf"][e]).T
        if c["fc"] == 1:
            g, u = y[:, :F], y[:, F:]
            y = g / (1.0 + torch.exp(-g)) * u * s["prob"][lo:hi, None]
        out[lo:hi] = y
    if not c["q"]:
        return {"out": out.to(torch.bfloat16)}
    q, sf = _quantize(out)
    return {"q": q, "sf": sf}


def _order(idx):
    """The (token, slot) pairs by expert, tokens ascending, and each pair's place."""
    order = torch.sort(idx.reshape(-1), stable=True)[1]
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    return order, place.view(idx.shape)


def _plain_sort(s):
    E, K, i32 = s["case"]["E"], s["case"]["K"], torch.int32
    order, place = _order(s["idx"])
    token = order // K
    counts = torch.bincount(s["idx"].reshape(-1), minlength=E)
    offsets = torch.cat([torch.zeros_like(counts[:1]), torch.cumsum(counts, 0)])
    return {"q": s["x_q"][token], "sf": s["x_sf"][token], "counts": counts.to(i32), "offsets": offsets.to(i32),
            "dst_row": place.to(i32), "src_token": token.to(i32), "perm_prob": s["prob"].reshape(-1)[order]}


def _plain_sort_bwd(s):
    place = s["dst_row"].long()
    dy = s["dy"].float()
    dprob = (dy[:, None, :] * s["y_perm"][place].float()).sum(2)
    dy_perm = torch.empty(s["y_perm"].shape, device="cuda")
    dy_perm[place] = s["prob"][:, :, None] * dy[:, None, :]
    return {"dy_perm": dy_perm.to(s["dy"].dtype), "dprob": dprob}


def _plain_quant_w(s):
    c = s["case"]
    G, N, K = c["groups"], c["rows"], c["cols"]
    q, sf = _quantize_blocks(s["x"].float().view(G * N, K))
    out = {"q": q.view(G, N, K), "sf": sf.view(G, N // BLOCK, K // BLOCK)}
    if c["both"]:
        out["q_t"], out["sf_t"] = out["q"].transpose(1, 2).contiguous(), out["sf"].transpose(1, 2).contiguous()
    return out


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "quant":
        out = dict(zip(("q", "sf"), _quantize(state["x"].float())))
    else:
        out = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "quant_w": _plain_quant_w, "product": _plain_product,
               "sort": _plain_sort, "sort_bwd": _plain_sort_bwd}[op](state)
    return _named(out, *out)


# ---- work --------------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    eb = 4 if c.get("dtype") == "f32" else 2
    if op == "norm":
        per = eb * (1 + 2 * c["res"] + c["y"]) + (1 + 4 / BLOCK) * c["q"]
        return {"bytes": c["rows"] * (c["h"] * per + 4) + 4 * c["h"], "flops": 6 * c["rows"] * c["h"]}
    if op == "norm_bwd":
        return {"bytes": c["rows"] * (c["h"] * eb * (3 + c["res"]) + 4) + 8 * c["h"],
                "flops": 10 * c["rows"] * c["h"]}
    if op == "quant":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (2 + 1 + 4 / BLOCK), "flops": 2 * n}
    if op == "quant_w":
        n = c["groups"] * c["rows"] * c["cols"]
        return {"bytes": n * (2 + (1 + 4 / BLOCK ** 2) * (1 + c["both"])), "flops": 2 * n}
    T, h, E, K = c["T"], c["h"], c["E"], c["K"]
    P = T * K
    if op == "product":
        F = c["F"]
        kd, n = (h, 2 * F) if c["fc"] == 1 else (F, h)
        # experts that any token needs: a token's K are distinct; skewed shares leave
        # fewer of E busy than even ones would (E P / (P + E - 1) for exponential shares)
        busy = min(E, max(K, E * P / (P + E - 1)))
        b = busy * n * kd * (1 + 4 / BLOCK ** 2) + P * kd * (1 + 4 / BLOCK)
        b += P * (F if c["fc"] == 1 else h) * (1 + 4 / BLOCK if c["q"] else 2)
        return {"bytes": b, "flops": 2 * P * kd * n}
    if op == "sort":
        return {"bytes": (T + P) * h * (1 + 4 / BLOCK) + P * 24 + 8 * E, "flops": 0}
    return {"bytes": (T + 2 * P) * h * eb + P * 12, "flops": 3 * P * h}


# ---- the definitions in 64 bits ----------------------------------------------------------------
def _e4m3_table():
    """The 127 magnitudes of E4M3 in order of their codes: subnormals, then 2^(e - 7) (1 + m / 8)."""
    m = torch.arange(127, device="cuda")
    e, f = m // 8, (m % 8).double()
    return torch.where(e == 0, f * 2.0 ** -9, torch.exp2(e.double() - 7) * (1 + f / 8))


def _nearest(v):
    """The nearest E4M3 number of 64-bit values, ties to the even code; beyond the largest, the largest.
    (A tie of 64-bit quotients of 16-bit numbers is within 2^-50 of the border, and nothing else is.)"""
    table = _e4m3_table()
    mid = (table[1:] + table[:-1]) / 2
    a = v.abs()
    lo = torch.searchsorted(mid, a)                # midpoints below a: a tie is left to the lower code
    lo = lo - ((lo > 0) & (a <= mid[(lo - 1).clamp(min=0)] * (1 + 2.0 ** -50))).long()
    tie = (lo < mid.numel()) & (a >= mid[lo.clamp(max=mid.numel() - 1)] * (1 - 2.0 ** -50))
    return torch.copysign(table[lo + (tie & (lo % 2 == 1)).long()], v)


def _exact_rows(v):
    q, sf = torch.empty_like(v), torch.empty(v.shape[0], v.shape[1] // BLOCK, dtype=torch.float64, device="cuda")
    for lo in range(0, v.shape[0], 4096):
        b = v[lo:lo + 4096].unflatten(1, (-1, BLOCK))
        top = b.abs().max(2)[0]
        q[lo:lo + 4096] = _nearest(b * TOP / top.unsqueeze(2)).flatten(1)
        sf[lo:lo + 4096] = top / TOP
    return q, sf


def _decode64(q, sf, tall):
    """float64 values of codes whose scale (of a row, or of 128 of them) covers 128 columns."""
    m = (q & 127).long()
    v = torch.where(q >= 128, -_e4m3_table()[m], _e4m3_table()[m])
    r = torch.arange(q.shape[0], device="cuda") // (BLOCK if tall else 1)
    k = torch.arange(q.shape[1], device="cuda") // BLOCK
    return v * sf.double()[r[:, None], k[None, :]]


def exact(case, seed):
    c, op, s = case, case["op"], prepare(case, seed)
    if op == "norm":
        v = s["x"].double()
        v = v if s["res"] is None else v + s["res"].double()
        rms = torch.sqrt(v.pow(2).sum(1) / c["h"] + EPS)
        y = v / rms[:, None] * s["w"].double()
        out = {"rstd": 1 / rms}
        if c["res"]:
            out["sum"] = v
        if c["y"]:
            out["y"] = y
        if c["q"]:
            out["q"], out["sf"] = _exact_rows(y)
        return out
    if op == "norm_bwd":
        v, r = s["sum"].double(), s["rstd"].double()[:, None]
        dy, w = s["dy"].double(), s["w"].double()
        # y = v r w with r = (mean v^2 + eps)^(-1/2): dr/dv = -r^3 v / h
        dr = (dy * w * v).sum(1, keepdim=True)
        dx = dy * w * r - v * r.pow(3) * dr / c["h"]
        return {"dx": dx if s["dsum"] is None else dx + s["dsum"].double(), "dw": (dy * v * r).sum(0)}
    if op == "quant":
        return dict(zip(("q", "sf"), _exact_rows(s["x"].double())))
    if op == "quant_w":
        G, N, K = c["groups"], c["rows"], c["cols"]
        q, sf = (torch.empty(t.shape, dtype=torch.float64, device="cuda") for t in (s["q"], s["sf"]))
        for g in range(G):
            b = s["x"][g].double().unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK)).transpose(1, 2)
            top = b.abs().flatten(2).max(2)[0]
            q[g] = _nearest(b * TOP / top[:, :, None, None]).transpose(1, 2).flatten(2).flatten(0, 1)
            sf[g] = top / TOP
        out = {"q": q, "sf": sf}
        if c["both"]:
            out["q_t"], out["sf_t"] = q.mT.contiguous(), sf.mT.contiguous()
        return out
    if op == "product":
        F = c["F"]
        out = torch.zeros(c["T"] * c["K"], F if c["fc"] == 1 else c["h"], dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            lo, hi = s["bounds"][e], s["bounds"][e + 1]
            if hi > lo:
                z = _decode64(s["a_q"][lo:hi], s["a_sf"][lo:hi], False) @ _decode64(s["w_q"][e], s["w_sf"][e], True).T
                if c["fc"] == 1:
                    z = z[:, :F] * torch.sigmoid(z[:, :F]) * z[:, F:] * s["prob"][lo:hi, None].double()
                out[lo:hi] = z
        return dict(zip(("q", "sf"), _exact_rows(out))) if c["q"] else {"out": out}
    if op == "sort":
        h = s["idx"].cpu().numpy()
        pairs = sorted((int(e), t, k) for t, row in enumerate(h) for k, e in enumerate(row))
        token = torch.tensor([t for _, t, _ in pairs], device="cuda")
        slot = torch.tensor([k for _, _, k in pairs], device="cuda")
        table = torch.cat([_e4m3_table(), torch.full((1,), math.nan, dtype=torch.float64, device="cuda")])
        x = torch.where(s["x_q"] >= 128, -1.0, 1.0).double() * table[(s["x_q"] & 127).long()]
        return {"q": x[token], "sf": s["x_sf"].double()[token], "counts": None, "offsets": None, "dst_row": None,
                "src_token": None, "perm_prob": s["prob"].double()[token, slot]}
    T, K = c["T"], c["K"]
    dy, p = s["dy"].double(), s["prob"].double()
    dy_perm = torch.zeros(s["y_perm"].shape, dtype=torch.float64, device="cuda")
    dprob = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for k in range(K):
        to = s["dst_row"][:, k].long()
        dy_perm[to] = p[:, k, None] * dy
        dprob[:, k] = torch.einsum("th,th->t", dy, s["y_perm"][to].double())
    return {"dy_perm": dy_perm, "dprob": dprob}
