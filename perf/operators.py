"""Timed cases of the serving operators: MXFP4 quantisation, the grouped expert
products on MXFP4 operands, and the whole MoE layer for a few tokens with bf16
and with MXFP4 expert weights.

Every case gives the operator's plain form (elementary torch operations, sums
in 32 bits, the routing's keys in 64) and, with ``own`` set, the framework's
call on the same inputs.  Inputs are made from the seed alone: activations
N(0, 1), expert weights N(0, 1/fan-in), router weights N(0, 0.02^2), the
workloads' own distributions.
"""

import math

import numpy as np
import torch

own = False

SWIGLU, GELU = "swiglu", "gelu"
SOFTMAX, SIGMOID = "softmax", "sigmoid"


# ---- cases ------------------------------------------------------------------------
def _quant(name, rows, cols, groups, ragged):
    return {"name": name, "op": "quant", "rows": rows, "cols": cols, "groups": groups, "ragged": ragged}


def _product(name, fc, T, h, E, K, F):
    return {"name": name, "op": "product", "fc": fc, "T": T, "h": h, "E": E, "K": K, "F": F}


def _few(name, op, T, h, E, K, F, score=SOFTMAX, act=SWIGLU, bias=False, shared=0):
    return {"name": name, "op": op, "T": T, "h": h, "E": E, "K": K, "F": F, "score": score,
            "act": act, "bias": bias, "shared": shared}


def listed():
    return [
        # the activations of one decoding step before the experts: latency
        _quant("quant_33x2048", 33, 2048, 64, True),
        # a permuted prefill batch (8192 tokens, top-2), ragged experts
        _quant("quant_16384x4096", 16384, 4096, 8, True),
        # loading: the first projections of 8 experts, uniform groups
        _quant("quant_weights", 8 * 28672, 4096, 8, False),
        # a prefill batch of the 8-expert layer, compute bound
        _product("fc1_T8192_E8", 1, 8192, 4096, 8, 2, 14336),
        # a chunk of a fine-grained layer, ~128 rows an expert, between the two bounds
        _product("fc2_T512_E32", 2, 512, 7168, 32, 8, 2048),
        # a small batch over many experts: odd counts, empty experts, weights bound
        _product("fc1_T61_E64", 1, 61, 2048, 64, 8, 1024),
        # one sequence decoding on a small layer: latency
        _few("few_T1_E64", "few", 1, 2048, 64, 8, 1024),
        # a small decoding batch of the sigmoid-routed layer with a shared expert
        _few("few_T5_E256", "few", 5, 7168, 256, 8, 2048, score=SIGMOID, shared=1),
        # a larger decoding batch where every expert is busy
        _few("few_T32_E8", "few", 32, 4096, 8, 2, 14336),
        # the same three regimes with 4-bit expert weights
        _few("few4_T1_E256", "few4", 1, 7168, 256, 8, 2048, score=SIGMOID, shared=1),
        _few("few4_T13_E8", "few4", 13, 4096, 8, 2, 14336),
        _few("few4_T64_E64", "few4", 64, 2048, 64, 8, 1024),
    ]


def _log(rng, lo, hi, step):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def _unnamed(c):
    return {k: v for k, v in c.items() if k != "name"}


def draw(rng):
    op = rng.choice(["quant", "product", "few", "few4"])
    if op == "quant":
        cols = _log(rng, 128, 7168, 128)
        groups = rng.choice([1, 3, 8, 64, 256])
        if rng.random() < 0.3:  # uniform groups of whole 128-row tiles or not
            rows = groups * _log(rng, 1, max(2, min(28672, 100_000_000 // (groups * cols))), 1)
            return _unnamed(_quant("", rows, cols, groups, False))
        rows = _log(rng, 1, max(2, min(65536, 400_000_000 // cols)), 1)
        return _unnamed(_quant("", rows, cols, groups, True))
    E = rng.choice([4, 8, 32, 64, 128, 256])
    K = rng.choice([k for k in (1, 2, 6, 8) if k <= E])
    h = _log(rng, 512, 7168, 128)
    F = _log(rng, 256, 14336, 128)
    if op == "product":
        F = min(F, max(256, 600_000_000 // (E * h) // 128 * 128))
        T = _log(rng, 1, 8192, 1)
        T = max(1, min(T, int(1.5e12 // (4 * K * h * F))))
        return _unnamed(_product("", rng.choice([1, 2]), T, h, E, K, F))
    F = min(F, max(256, 1_500_000_000 // (E * h) // 128 * 128))
    T = _log(rng, 1, 64, 1)
    T = max(1, min(T, int(1.0e12 // (8 * h * F * 3))))
    act, bias, shared = SWIGLU, False, rng.choice([0, 0, 1])
    if op == "few" and rng.random() < 0.25:
        act, bias, shared = GELU, rng.random() < 0.5, 0
    if op == "few" and rng.random() < 0.5:  # 16-byte rows are enough for bf16 weights
        h, F = h - 8 * rng.randrange(1, 8), F - 8 * rng.randrange(1, 8)
    return _unnamed(_few("", op, T, h, E, K, F, rng.choice([SOFTMAX, SIGMOID]), act, bias, shared))


# ---- inputs -----------------------------------------------------------------------
def _gen(seed, tag):
    return torch.Generator(device="cuda").manual_seed(1_000_003 * int(seed) + tag)


def _normal(shape, std, seed, tag, dtype=torch.bfloat16):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, std, generator=_gen(seed, tag))


def _offsets(rows, groups, seed):
    """Ragged group boundaries [groups + 1] that cover the rows: a skewed split,
    with groups of no rows where there are more groups than rows."""
    r = np.random.default_rng(int(seed))
    w = r.dirichlet(np.full(groups, 1.0))
    return np.concatenate([[0], np.cumsum(r.multinomial(rows, w))]).astype(np.int32)


def _row_slots(offsets, rows, groups):
    """Where each row's scales lie: its tile of 128 rows (numbered group after
    group) times 128 plus its row within the tile."""
    if offsets is None:
        n = rows // groups
        r = torch.arange(rows, device="cuda")
        g, lr = r // n, r % n
        return (g * ((n + 127) // 128)) * 128 + lr
    off = torch.from_numpy(offsets.astype(np.int64)).cuda()
    tiles = (off[1:] - off[:-1] + 127) // 128
    first = torch.cumsum(tiles, 0) - tiles
    r = torch.arange(rows, device="cuda")
    g = torch.searchsorted(off, r, right=True) - 1
    return first[g] * 128 + (r - off[g])


def _to_atoms(scales, slots, tiles):
    """Scale codes [rows, cols / 32] -> the 512-byte atoms of 128 rows x 128
    columns: row i, block j at byte 16 (i % 32) + 4 (i / 32) + j."""
    kb = scales.shape[1] // 4
    flat = torch.zeros(tiles * 128, kb * 4, dtype=torch.uint8, device="cuda")
    flat[slots] = scales
    return flat.view(tiles, 4, 32, kb, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _from_atoms(atoms, tiles, kb):
    """The reverse: [tiles * 128, cols / 32] scale codes."""
    a = atoms[: tiles * kb * 512].view(tiles, kb, 32, 4, 4)
    return a.permute(0, 3, 2, 1, 4).reshape(tiles * 128, kb * 4)


def _tiles(rows, groups):
    return (rows + 127) // 128 + groups


def _quantize(x):
    """bf16 [rows, cols] -> 4-bit codes, two a byte (even column in the low
    half), and scale codes [rows, cols / 32]: X = floor(log2 max|x|) - 2, values
    x / 2^X to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    rows, cols = x.shape
    v = x.float().view(rows, cols // 32, 32)
    amax = v.abs().amax(2)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 1, torch.full_like(amax, -200, dtype=torch.int32))
    code = (e - 2 + 127).clamp(0, 254)
    y = torch.ldexp(v.abs(), (127 - code).unsqueeze(2))
    mag = ((y > 0.25).int() + (y >= 0.75).int() + (y > 1.25).int() + (y >= 1.75).int()
           + (y > 2.5).int() + (y >= 3.5).int() + (y > 5.0).int())
    c = (mag + 8 * torch.signbit(v).int()).view(rows, cols // 2, 2)
    return (c[:, :, 0] + 16 * c[:, :, 1]).to(torch.uint8), code.to(torch.uint8)


def _values(q, scales, dtype=torch.float32):
    """The values that codes [..., cols / 2] and scale codes [..., cols / 32] stand for."""
    c = torch.stack([q & 15, q >> 4], -1).flatten(-2)
    mag = (c & 7).to(dtype)
    v = torch.where(mag < 4, mag * 0.5, torch.where(mag < 6, mag - 2, mag * 2 - 8))
    v = torch.where(c >= 8, -v, v)
    s = torch.ldexp(torch.ones((), dtype=dtype, device=q.device), scales.to(torch.int32) - 127)
    return (v.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def _quantized_weights(E, rows, cols, std, seed, tag):
    """Codes [E, rows, cols / 2] and scale atoms of E weight matrices, one expert at a time."""
    q = torch.empty(E, rows, cols // 2, dtype=torch.uint8, device="cuda")
    kb, n = cols // 128, rows // 128
    sf = torch.zeros(_tiles(E * rows, E) * kb * 512, dtype=torch.uint8, device="cuda")
    g = _gen(seed, tag)
    w = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(rows, device="cuda")
    for e in range(E):
        q[e], s = _quantize(w.normal_(0.0, std, generator=g))
        sf[e * n * kb * 512:(e + 1) * n * kb * 512] = _to_atoms(s, slots, n)
    return q, sf


def _keys(x, w_r, sel_bias, score):
    logits = x.double() @ w_r.double().T
    key = torch.sigmoid(logits).float() if score == SIGMOID else logits.float()
    return logits, key if sel_bias is None else key + sel_bias


def _tokens(c, w_r, sel_bias, seed):
    """Activations whose routing is decided: a token with two keys of its best
    K + 1 nearer than 1e-5 (the last bits of a sum would choose) is drawn anew."""
    x = _normal((c["T"], c["h"]), 1.0, seed, 1)
    for k in range(20):
        key = _keys(x, w_r, sel_bias, c["score"])[1]
        best = torch.sort(key, dim=1, descending=True)[0][:, : c["K"] + 1]
        near = (best[:, :-1] - best[:, 1:] < 1e-5).any(1)
        x = torch.where(near[:, None], _normal(x.shape, 1.0, seed, 100 + k), x)
    return x


def prepare(case, seed):
    c = case
    if c["op"] == "quant":
        rows, cols, groups = c["rows"], c["cols"], c["groups"]
        off = _offsets(rows, groups, seed) if c["ragged"] else None
        x = _normal((rows, cols), 1.0 if c["ragged"] else 1.0 / math.sqrt(cols), seed, 1)
        return {"case": c, "x": x, "offsets": None if off is None else torch.from_numpy(off).cuda(),
                "q": torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda"),
                "sf": torch.empty(_tiles(rows, groups) * (cols // 128) * 512, dtype=torch.uint8, device="cuda"),
                "out": torch.empty_like(x)}
    T, h, E, K, F = c["T"], c["h"], c["E"], c["K"], c["F"]
    P = T * K
    if c["op"] == "product":
        kd, n = (h, 2 * F) if c["fc"] == 1 else (F, h)
        off = _offsets(P, E, seed)
        a_q, s = _quantize(_normal((P, kd), 1.0, seed, 1))
        slots = _row_slots(off, P, E)
        tiles = _tiles(P, E)
        a_sf = _to_atoms(s, slots, tiles)
        n_pad = (n + 127) // 128 * 128  # h and F are multiples of 128
        w_q, w_sf = _quantized_weights(E, n_pad, kd, 1.0 / math.sqrt(kd), seed, 2)
        prob = torch.rand(P, device="cuda", generator=_gen(seed, 3)) if c["fc"] == 1 else None
        return {"case": c, "a_q": a_q, "a_sf": a_sf, "slots": slots, "tiles": tiles, "w_q": w_q,
                "w_sf": w_sf, "prob": prob, "offsets": torch.from_numpy(off).cuda(),
                "bounds": off.tolist(),
                "out": torch.empty(P, F if c["fc"] == 1 else h, dtype=torch.bfloat16, device="cuda")}
    r1 = 2 * F if c["act"] == SWIGLU else F
    s = {"case": c, "w_r": _normal((E, h), 0.02, seed, 2, torch.float32),
         "sel_bias": _normal((E,), 0.1, seed, 3, torch.float32) if c["score"] == SIGMOID else None}
    s["x"] = _tokens(c, s["w_r"], s["sel_bias"], seed)
    std1, std2, ns = 1.0 / math.sqrt(h), 1.0 / math.sqrt(F), c["shared"]
    if c["op"] == "few":
        s["w1"], s["w2"] = _normal((E, r1, h), std1, seed, 4), _normal((E, h, F), std2, seed, 5)
        s["b1"] = _normal((E, r1), std1, seed, 6) if c["bias"] else None
        s["b2"] = _normal((E, h), std2, seed, 7) if c["bias"] else None
        s["w1s"] = _normal((r1, h), std1, seed, 8) if ns else None
        s["w2s"] = _normal((h, F), std2, seed, 9) if ns else None
    else:
        s["w1"], s["w1_sf"] = _quantized_weights(E, r1, h, std1, seed, 4)
        s["w2"], s["w2_sf"] = _quantized_weights(E, h, F, std2, seed, 5)
        s["w1s"], s["w1s_sf"] = _quantized_weights(1, r1, h, std1, seed, 8) if ns else (None, None)
        s["w2s"], s["w2s_sf"] = _quantized_weights(1, h, F, std2, seed, 9) if ns else (None, None)
    s["y"] = torch.empty(T, h, dtype=torch.bfloat16, device="cuda")
    s["idx"] = torch.empty(T, K, dtype=torch.int32, device="cuda")
    s["prob"] = torch.empty(T, K, dtype=torch.float32, device="cuda")
    return s


# ---- the framework's calls --------------------------------------------------------------
def _plan(M, s):
    """The config and workspace that a serving program makes once per layer and batch size."""
    c = s["case"]
    cfg = M.make_config(c["T"], c["h"], c["E"], c["K"], c["F"],
                        score=M.MOE_SCORE_SIGMOID if c.get("score") == SIGMOID else M.MOE_SCORE_SOFTMAX,
                        act=M.MOE_ACT_GELU if c.get("act") == GELU else M.MOE_ACT_SWIGLU,
                        has_bias=int(c.get("bias", False)), n_shared=c.get("shared", 0))
    ws = torch.empty(M.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda") if c["op"] != "product" else None
    s["plan"] = cfg, ws
    return s["plan"]


def _run_own(s):
    from mixture_experts_layer_softmax_gb300 import moe as M
    c = s["case"]
    if c["op"] == "quant":
        M.moe_mxfp4_quantize(c["rows"], c["cols"], c["groups"], s["offsets"], s["x"], s["q"], s["sf"])
        M.moe_mxfp4_dequantize(c["rows"], c["cols"], c["groups"], s["offsets"], s["q"], s["sf"], s["out"])
        return s["out"]
    cfg, ws = s.get("plan") or _plan(M, s)
    if c["op"] == "product":
        if c["fc"] == 1:
            M.moe_expert_fc1_mxfp4(cfg, s["a_q"], s["a_sf"], s["offsets"], s["prob"], s["w_q"], s["w_sf"],
                                   s["out"], None, None)
        else:
            M.moe_expert_fc2_mxfp4(cfg, s["a_q"], s["a_sf"], s["offsets"], s["w_q"], s["w_sf"], s["out"])
        return s["out"]
    if c["op"] == "few":
        M.moe_layer_fwd_few(cfg, s["x"], s["w_r"], None, s["sel_bias"], s["w1"], s["b1"], s["w2"], s["b2"],
                            s["w1s"], s["w2s"], s["y"], s["idx"], s["prob"], ws)
    else:
        M.moe_layer_fwd_few_mxfp4(cfg, s["x"], s["w_r"], None, s["sel_bias"], s["w1"], s["w1_sf"], s["w2"],
                                  s["w2_sf"], s["w1s"], s["w1s_sf"], s["w2s"], s["w2s_sf"], s["y"], s["idx"],
                                  s["prob"], ws)
    return {"y": s["y"], "idx": s["idx"], "prob": s["prob"]}


# ---- the plain forms -----------------------------------------------------------------------
def _act(hidden, act, F):
    if act == GELU:
        return 0.5 * hidden * (1 + torch.erf(hidden * math.sqrt(0.5)))
    g, u = hidden[..., :F], hidden[..., F:]
    return g / (1 + torch.exp(-g)) * u


def _plain_product(s):
    c = s["case"]
    kb = s["a_q"].shape[1] * 2 // 128
    x = _values(s["a_q"], _from_atoms(s["a_sf"], s["tiles"], kb)[s["slots"]])
    E, n, _ = s["w_q"].shape
    scales = _from_atoms(s["w_sf"], E * n // 128, kb).view(E, n, kb * 4)
    for e, (lo, hi) in enumerate(zip(s["bounds"][:-1], s["bounds"][1:])):
        if hi > lo:
            y = x[lo:hi] @ _values(s["w_q"][e], scales[e]).T
            if c["fc"] == 1:
                y = _act(y, SWIGLU, c["F"]) * s["prob"][lo:hi, None]
            s["out"][lo:hi] = y
    return s["out"]


def _plain_weights(s, name, pick):
    """The chosen experts' matrices in 32 bits."""
    w = s[name]
    if s["case"]["op"] == "few":
        return (w if w.dim() == 2 else w[pick]).float()
    E, n, half = w.shape
    kb = half * 2 // 128
    scales = _from_atoms(s[name + "_sf"], E * n // 128, kb).view(E, n, kb * 4)
    return _values(w[pick], scales[pick])


def _plain_layer(s):
    c, x = s["case"], s["x"].float()
    T, K, F = c["T"], c["K"], c["F"]
    logits, key = _keys(s["x"], s["w_r"], s["sel_bias"], c["score"])
    idx = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :K]
    score = torch.sigmoid(logits) if c["score"] == SIGMOID else torch.exp(logits - logits.amax(1, True))
    p = score.gather(1, idx)
    p = (p / p.sum(1, True)).float()
    y = torch.zeros(T, c["h"], device=x.device)
    for k in range(K):  # slot by slot: each token's k-th expert
        e = idx[:, k]
        hid = torch.bmm(_plain_weights(s, "w1", e), x.unsqueeze(2)).squeeze(2)
        a = _act(hid + s["b1"][e].float() if c["bias"] else hid, c["act"], F)
        o = torch.bmm(_plain_weights(s, "w2", e), a.unsqueeze(2)).squeeze(2)
        y += p[:, k:k + 1] * (o + s["b2"][e].float() if c["bias"] else o)
    if c["shared"]:
        w1, w2 = (_plain_weights(s, n, 0).view(-1, w) for n, w in (("w1s", c["h"]), ("w2s", F)))
        y += _act(x @ w1.T, c["act"], F) @ w2.T
    return {"y": y.to(torch.bfloat16), "idx": idx.to(torch.int32), "prob": p}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "quant":
        q, code = _quantize(state["x"])
        return _values(q, code).to(torch.bfloat16)
    return _plain_product(state) if op == "product" else _plain_layer(state)


# ---- work --------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "quant":
        # read bf16, write codes and scales, read them, write the values
        n = c["rows"] * c["cols"]
        return {"bytes": n * (2 + 2 * (0.5 + 1 / 32) + 2), "flops": 4 * n}
    T, h, E, K, F = c["T"], c["h"], c["E"], c["K"], c["F"]
    P = T * K
    if c["op"] == "product":
        kd, n = (h, 2 * F) if c["fc"] == 1 else (F, h)
        # a skewed split leaves some experts without rows when rows are few:
        # of E exponential shares, P draws reach E P / (P + E - 1) on average
        busy = E * P / (P + E - 1)
        b = (busy * n + P) * kd * (0.5 + 1 / 32) + P * (F if c["fc"] == 1 else h) * 2
        return {"bytes": b, "flops": 2 * P * kd * n}
    r1 = 2 * F if c["act"] == SWIGLU else F
    busy = E * (1 - (1 - K / E) ** T) + c["shared"]  # experts that any token needs
    per = 2 if c["op"] == "few" else 0.5 + 1 / 32
    b = busy * (r1 + F) * h * per + E * h * 4 + T * h * 4 + P * 8
    return {"bytes": b, "flops": 2 * T * ((K + c["shared"]) * (r1 + F) * h + E * h)}


# ---- the definitions in 64 bits ----------------------------------------------------------------
_LADDER = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _decode64(q, sf, slot, cols):
    """float64 [rows, cols] of codes [rows, cols / 2] whose row r has its scales
    at place slot[r] of the tiles, straight from the format's byte addresses."""
    table = torch.tensor(_LADDER + tuple(-v for v in _LADDER), dtype=torch.float64, device=q.device)
    v = torch.empty(q.shape[0], cols, dtype=torch.float64, device=q.device)
    v[:, 0::2] = table[(q & 15).long()]
    v[:, 1::2] = table[(q >> 4).long()]
    tile, i = slot // 128, slot % 128
    b = torch.arange(cols // 32, device=q.device)
    at = ((tile * (cols // 128))[:, None] + b // 4) * 512 + (16 * (i % 32) + 4 * (i // 32))[:, None] + b % 4
    scale = torch.exp2(sf[at].double() - 127)
    return v * scale.repeat_interleave(32, 1)


def _exact_quant(x):
    """The nearest value of the ladder by distance, ties to the even place."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for lo in range(0, x.shape[0], 8192):
        v = x[lo:lo + 8192].double().view(-1, x.shape[1] // 32, 32)
        amax = v.abs().amax(2, True)
        power = torch.where(amax > 0, torch.floor(torch.log2(amax)) - 2, torch.full_like(amax, -127.0)).clamp(min=-127)
        y = v.abs() * torch.exp2(-power)
        best, best_d = torch.zeros_like(y), y.clone()
        for n, w in list(enumerate(_LADDER))[1:]:
            d = (y - w).abs()
            nearer = (d < best_d) | ((d == best_d) & (n % 2 == 0))
            best, best_d = torch.where(nearer, torch.full_like(y, w), best), torch.where(nearer, d, best_d)
        out[lo:lo + 8192] = (torch.copysign(best, v) * torch.exp2(power)).view(-1, x.shape[1])
    return out


def _ffn64(x, w1, w2, b1, b2, act, F):
    z = x @ w1.T
    z = z if b1 is None else z + b1.double()
    if act == GELU:
        a = z * torch.special.ndtr(z)
    else:
        a = z[:, :F] * torch.sigmoid(z[:, :F]) * z[:, F:]
    o = a @ w2.T
    return o if b2 is None else o + b2.double()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quant":
        return _exact_quant(s["x"])
    T, h, E, K, F = c["T"], c["h"], c["E"], c["K"], c["F"]
    if c["op"] == "product":
        kd = s["a_q"].shape[1] * 2
        n = s["w_q"].shape[1]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for e in range(E):
            lo, hi = s["bounds"][e], s["bounds"][e + 1]
            if hi == lo:
                continue
            w = _decode64(s["w_q"][e], s["w_sf"], torch.arange(n, device="cuda") + e * n, kd)
            z = _decode64(s["a_q"][lo:hi], s["a_sf"], s["slots"][lo:hi], kd) @ w.T
            if c["fc"] == 1:
                z = z[:, :F] * torch.sigmoid(z[:, :F]) * z[:, F:] * s["prob"][lo:hi, None].double()
            out[lo:hi] = z
        return out
    r1 = 2 * F if c["act"] == SWIGLU else F
    x = s["x"].double()
    logits = x @ s["w_r"].double().T
    scores = 1 / (1 + torch.exp(-logits)) if c["score"] == SIGMOID else torch.softmax(logits, 1)
    key = scores.float().double() + s["sel_bias"].double() if c["score"] == SIGMOID else logits
    idx = torch.argsort(key, dim=1, descending=True, stable=True)[:, :K]
    p = torch.take_along_dim(scores, idx, 1)
    p = p / p.sum(1, True)
    y = torch.zeros(T, h, dtype=torch.float64, device="cuda")

    def matrix(name, e, rows, cols):
        w = s[name]
        if c["op"] == "few":
            return (w if w.dim() == 2 else w[e]).double()
        return _decode64(w[e], s[name + "_sf"], torch.arange(rows, device="cuda") + e * rows, cols)

    for e in torch.unique(idx).tolist():
        t, k = torch.nonzero(idx == e, as_tuple=True)
        o = _ffn64(x[t], matrix("w1", e, r1, h), matrix("w2", e, h, F),
                   s["b1"][e] if c["bias"] else None, s["b2"][e] if c["bias"] else None, c["act"], F)
        y.index_add_(0, t, o * p[t, k][:, None])
    if c["shared"]:
        y += _ffn64(x, matrix("w1s", 0, r1, h), matrix("w2s", 0, h, F), None, None, c["act"], F)
    return {"y": y, "idx": None, "prob": p}
