"""The 8-bit operators of 2:4-masked weights, as cases to measure: what each
computes in elementary torch operations (the plain form), the calls a user
makes of this package for the same result, and the result from the definition
in 64 bits.

Format of the 8-bit operands.  Values are e4m3; the scale of a block is 2^s,
held as the byte s + 127 (e8m0), where s is the least integer >= -127 with
amax <= 448 * 2^s for the largest finite magnitude amax of the block (s = 0 for
a block of zeros).  Dense operands have blocks of 1 x 128 along their rows and
scales [blocks][rows]; 2:4 operands have blocks of 128 x 128, two values for
each aligned group of four along a row, and a 32-bit word of positions for each
32 entries (4 bits a group: first position, then second).  Rows are padded with
zeros to whole blocks of 128.

Operators (the "op" of a case):
  quant     activations or gradients to 8 bits along the rows, the columns or both
  compress  a weight matrix under a 2:4 mask to 8 bits, as W, W^T or both
  linear    Y = X A^T with a 2:4 operand A (A = W: forward; A = W^T: data gradient)
  wgrad     dW = dY^T X, kept where the 2:4 mask keeps W
  moe       a mixture-of-experts layer for a few tokens, all experts 2:4
"""
import math

import torch

own = False

PAIRS = (0x4, 0x8, 0xC, 0x9, 0xD, 0xE)  # (first | second << 2) of the six 2:4 patterns


def listed():
    return [
        # one token's activations before an 8-bit layer: latency
        {"name": "quant-1x4096", "op": "quant", "rows": 1, "cols": 4096, "dtype": "bf16", "along": "rows"},
        # a training step's activations, needed along features (forward) and along tokens (weight gradient)
        {"name": "quant-4096x11008-both", "op": "quant", "rows": 4096, "cols": 11008, "dtype": "bf16", "along": "both"},
        # a small fp32 layer, both orientations under its transposable mask
        {"name": "compress-1000x1028-f32", "op": "compress", "rows": 1000, "cols": 1028, "dtype": "f32", "along": "both"},
        # an MLP projection after a mask update
        {"name": "compress-11008x4096", "op": "compress", "rows": 11008, "cols": 4096, "dtype": "bf16", "along": "both"},
        # decoding: one token through an attention projection
        {"name": "linear-1x4096x4096", "op": "linear", "n": 1, "m": 4096, "k": 4096},
        # a ragged serving batch through an MLP projection
        {"name": "linear-37x11008x4096", "op": "linear", "n": 37, "m": 11008, "k": 4096},
        # a training step's MLP forward
        {"name": "linear-4096x11008x4096", "op": "linear", "n": 4096, "m": 11008, "k": 4096},
        # the data gradient through the largest matrix of the mask workloads (A = W^T)
        {"name": "linear-8192x28672x8192", "op": "linear", "n": 8192, "m": 28672, "k": 8192},
        # weight gradient of a small layer from an odd number of tokens
        {"name": "wgrad-1001x1024x1024", "op": "wgrad", "n": 1001, "m": 1024, "k": 1024},
        # a training step's MLP weight gradient
        {"name": "wgrad-4096x4096x11008", "op": "wgrad", "n": 4096, "m": 4096, "k": 11008},
        # decoding: one token through many small experts
        {"name": "moe-1-of-64x6", "op": "moe", "n": 1, "d": 2048, "f": 1408, "experts": 64, "topk": 6},
        # a decoding batch through few large experts
        {"name": "moe-33-of-16x4", "op": "moe", "n": 33, "d": 4096, "f": 2048, "experts": 16, "topk": 4},
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(("quant", "compress", "linear", "linear", "wgrad", "moe"))
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 32, 11008),
                "dtype": rng.choice(("bf16", "f32")), "along": rng.choice(("rows", "cols", "both"))}
    if op == "compress":
        return {"op": op, "rows": _log(rng, 64, 11008, 4), "cols": _log(rng, 64, 11008, 4),
                "dtype": rng.choice(("bf16", "f32")), "along": rng.choice(("rows", "cols", "both"))}
    if op == "linear":
        n = _log(rng, 1, 64) if rng.random() < 0.5 else _log(rng, 64, 8192)
        return {"op": op, "n": n, "m": _log(rng, 128, 11008, 4), "k": _log(rng, 128, 11008, 4)}
    if op == "wgrad":
        return {"op": op, "n": _log(rng, 64, 8192), "m": _log(rng, 128, 11008, 4),
                "k": _log(rng, 128, 11008, 4)}
    experts = rng.choice((4, 8, 16, 32, 64))
    return {"op": op, "n": _log(rng, 1, 64), "d": _log(rng, 512, 4096, 4), "f": _log(rng, 256, 2048, 4),
            "experts": experts, "topk": rng.randint(1, min(8, experts))}


def _up(v, q=128):
    return -(-v // q) * q


def _normal(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _operand24(gen, lead, rows, k):
    """A random 2:4 8-bit operand as compression of 0.02 * normal weights leaves it:
    two kept entries in each group of four, values over most of e4m3's range."""
    kp = _up(k)
    v = (82.0 * _normal(gen, *lead, rows, kp // 2)).clamp_(-448.0, 448.0)
    pairs = torch.tensor(PAIRS, device="cuda", dtype=torch.int64)
    nib = pairs[torch.randint(0, 6, (*lead, rows, kp // 4), device="cuda", generator=gen)]
    v[..., k // 2:] = 0.0
    nib[..., k // 4:] = 4
    word = (nib.reshape(*lead, rows, kp // 32, 8) << (4 * torch.arange(8, device="cuda"))).sum(-1)
    meta = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)
    s = torch.randint(114, 117, (*lead, _up(rows) // 128, kp // 128), device="cuda", generator=gen)
    return {"values": v.to(torch.float8_e4m3fn), "meta": meta,
            "scales": s.to(torch.uint8).view(torch.float8_e8m0fnu), "k": k}


def _mask24(gen, rows, cols):
    """A 2:4 mask whose 4 x 4 blocks hold two ones in every row and column (row pairs and
    their complements in a random order, columns shuffled), packed into 32-bit words."""
    base = torch.tensor([[1, 1, 0, 0], [0, 0, 1, 1]], device="cuda", dtype=torch.int64)
    br, bc = rows // 4, cols // 4
    order = torch.rand(br, bc, 4, device="cuda", generator=gen).argsort(-1)
    cols4 = torch.rand(br, bc, 4, device="cuda", generator=gen).argsort(-1)
    block = base[order % 2]  # [br, bc, 4 rows, 4 columns]
    block = block.gather(-1, cols4[:, :, None, :].expand(-1, -1, 4, -1))
    keep = block.permute(0, 2, 1, 3).reshape(rows, cols)
    keep = torch.nn.functional.pad(keep, (0, _up(cols, 32) - cols))
    word = (keep.reshape(rows, -1, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)


def _keep(mask, cols):
    bits = (mask.to(torch.int64)[..., None] >> torch.arange(32, device=mask.device)) & 1
    return bits.reshape(mask.shape[0], -1)[:, :cols].bool()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = dict(case)
    if op == "quant":
        # activations with a few loud features
        x = _normal(gen, case["rows"], case["cols"]) * torch.exp(_normal(gen, 1, case["cols"]))
        state["x"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    elif op == "compress":
        w = 0.02 * _normal(gen, case["rows"], case["cols"])
        state["w"] = w.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        state["mask"] = _mask24(gen, case["rows"], case["cols"])
    elif op == "linear":
        x = _normal(gen, case["n"], case["k"]) * torch.exp(0.5 * _normal(gen, 1, case["k"]))
        state["x"] = x.to(torch.bfloat16)
        state["a"] = _operand24(gen, (), case["m"], case["k"])
    elif op == "wgrad":
        state["x"] = _normal(gen, case["n"], case["k"]).to(torch.bfloat16)
        state["dy"] = (1e-3 * _normal(gen, case["n"], case["m"])).to(torch.bfloat16)
        state["mask"] = _mask24(gen, case["m"], case["k"])
    else:
        e, d, f = case["experts"], case["d"], case["f"]
        state["x"] = _normal(gen, case["n"], d).to(torch.bfloat16)
        state["router"] = (0.02 * _normal(gen, e, d)).to(torch.bfloat16)
        state["gate"] = _operand24(gen, (e,), f, d)
        state["up"] = _operand24(gen, (e,), f, d)
        state["down"] = _operand24(gen, (e,), d, f)
    return state


# ---- plain form: fp32 throughout -------------------------------------------

def _exponent(amax):
    """Least s >= -127 with amax <= 448 * 2^s (0 for amax = 0); 448 = 0.875 * 2^9."""
    m, p = torch.frexp(amax)
    s = torch.where(m <= 0.875, p - 9, p - 8).clamp(min=-127)
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _finite_abs(x):
    a = x.abs()
    return torch.where(torch.isfinite(a), a, torch.zeros_like(a))


def _times_pow2(x, s):
    """x * 2^s for -127 <= s <= 127, from the bits of 2^s (2^-127 is subnormal)."""
    bits = torch.where(s > -127, (s + 127) << 23, torch.full_like(s, 1 << 22))
    return x * bits.to(torch.int32).view(torch.float32)


def _e4m3(x):
    x = torch.where(torch.isfinite(x), x, torch.full_like(x, math.nan))
    return x.to(torch.float8_e4m3fn)


def _e8m0(s):
    return (s + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _quant_rows(x):
    """[r][c] -> e4m3 [r][cpad], exponents [r][cpad / 128]."""
    x = torch.nn.functional.pad(x.to(torch.float32), (0, _up(x.shape[1]) - x.shape[1]))
    b = x.reshape(x.shape[0], -1, 128)
    s = _exponent(_finite_abs(b).amax(-1))
    return _e4m3(_times_pow2(b, -s[..., None])).reshape(x.shape), s


def _dequant_rows(x):
    q, s = _quant_rows(x)
    b = q.to(torch.float32).reshape(q.shape[0], -1, 128)
    return _times_pow2(b, s[..., None]).reshape(q.shape)


def _expand24(a):
    """fp32 [..., rows, kpad] of a 2:4 operand."""
    v = a["values"].to(torch.float32)
    lead, kp = v.shape[:-1], 2 * v.shape[-1]
    g = torch.arange(8, device=v.device)
    nib = (a["meta"][..., None] >> (4 * g)) & 15
    pos = torch.stack((nib & 3, nib >> 2), -1).reshape(*lead, kp // 4, 2)
    v = v.reshape(*lead, kp // 4, 2)
    j = torch.arange(4, device=v.device)
    zero = torch.zeros((), device=v.device)
    dense = (torch.where(pos[..., :1] == j, v[..., :1], zero)
             + torch.where(pos[..., 1:] == j, v[..., 1:], zero)).reshape(*lead, kp)
    s = a["scales"].view(torch.uint8).to(torch.int32) - 127
    s = s.repeat_interleave(128, -2)[..., :lead[-1], :].repeat_interleave(128, -1)
    return _times_pow2(dense, s)


def _pack24(q, keep):
    """e4m3 [r][kpad] and kept entries -> values [r][kpad / 2], words [r][kpad / 32], groups
    with more than two kept."""
    r, kp = q.shape
    keep4 = torch.nn.functional.pad(keep, (0, kp - keep.shape[1])).reshape(r, kp // 4, 4)
    j = torch.arange(4, device=q.device)
    first = torch.where(keep4, j, j + 4).sort(-1).values[..., :2]  # kept positions, then unused ones
    count = keep4.sum(-1)
    p0 = torch.where(count > 0, first[..., 0], torch.zeros_like(count))
    other = torch.where(p0 == 3, 2, 3)
    p1 = torch.where(count > 1, first[..., 1], torch.where(count == 1, other, torch.ones_like(p0)))
    pos = torch.stack((p0, p1), -1)
    v = q.to(torch.float32).reshape(r, kp // 4, 4).gather(-1, pos)
    used = count[..., None] > torch.arange(2, device=q.device)
    v = torch.where(used, v, torch.zeros((), device=q.device)).reshape(r, kp // 2)
    nib = (p0 | (p1 << 2)).reshape(r, kp // 32, 8)
    word = (nib << (4 * torch.arange(8, device=q.device))).sum(-1)
    meta = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)
    return v.to(torch.float8_e4m3fn), meta, (count > 2).sum().to(torch.int32).reshape(1)


def _plain_quant(state):
    x, out = state["x"], {}
    if state["along"] in ("rows", "both"):
        q, s = _quant_rows(x)
        out["rows"] = (q, _e8m0(s).t().contiguous())
    if state["along"] in ("cols", "both"):
        q, s = _quant_rows(x.t())
        out["cols"] = (q, _e8m0(s).t().contiguous())
    return out


def _plain_compress(state):
    w, cols = state["w"].to(torch.float32), state["cols"]
    rows = w.shape[0]
    keep = _keep(state["mask"], cols)
    pad = (0, _up(cols) - cols, 0, _up(rows) - rows)
    kept = torch.nn.functional.pad(torch.where(keep, w, torch.zeros_like(w)), pad)
    b = kept.reshape(_up(rows) // 128, 128, _up(cols) // 128, 128)
    s = _exponent(_finite_abs(b).amax((1, 3)))
    q = _e4m3(_times_pow2(b, -s[:, None, :, None])).reshape(kept.shape)
    out = {}
    if state["along"] in ("rows", "both"):
        v, meta, bad = _pack24(q[:rows], keep)
        out["rows"] = (v, meta, _e8m0(s), bad)
    if state["along"] in ("cols", "both"):
        v, meta, bad = _pack24(q.view(torch.uint8).t()[:cols].contiguous().view(q.dtype), keep.t())
        out["cols"] = (v, meta, _e8m0(s.t().contiguous()), bad)
    return out


def _plain_linear(state):
    return (_dequant_rows(state["x"]) @ _expand24(state["a"]).t()).to(torch.bfloat16)


def _plain_wgrad(state):
    dw = _dequant_rows(state["dy"].t()) @ _dequant_rows(state["x"].t()).t()
    keep = _keep(state["mask"], state["k"])
    return torch.where(keep, dw, torch.zeros_like(dw)).to(torch.bfloat16)


def _route(x, router, topk, dtype):
    """Chosen experts [n][topk], largest logit first (ties to the lowest index), and their weights."""
    logits = x.to(torch.float64) @ router.to(torch.float64).t()
    top, ids = logits.sort(dim=-1, descending=True, stable=True)
    top, ids = top[:, :topk], ids[:, :topk]
    p = torch.exp((top - top[:, :1]).to(dtype))
    return ids, p / p.sum(-1, keepdim=True)


def _pick(a, ids):
    """The operands of some experts out of a stack."""
    part = lambda t: t.view(torch.uint8)[ids].view(t.dtype)
    return {"values": part(a["values"]), "meta": a["meta"][ids], "scales": part(a["scales"])}


def _plain_moe(state):
    x = state["x"]
    n, d, f, topk = state["n"], state["d"], state["f"], state["topk"]
    ids, w = _route(x, state["router"], topk, torch.float32)
    flat = ids.reshape(-1)
    parts = (state["gate"], state["up"], state["down"])
    if n * topk < state["experts"]:  # a few tokens: only the experts they chose
        gate, up, down = (_expand24(_pick(p, flat)) for p in parts)
        xs = x.to(torch.float32).repeat_interleave(topk, 0)[:, None, :]  # [n topk][1][d]
        g = xs @ gate[..., :d].transpose(1, 2).contiguous()
        h = g * torch.sigmoid(g) * (xs @ up[..., :d].transpose(1, 2).contiguous())
        y = (h @ down[..., :f].transpose(1, 2).contiguous()).reshape(n, topk, d)
        return (y * w[..., None]).sum(1).to(torch.bfloat16)
    gate, up, down = (_expand24(p) for p in parts)
    xs = x.to(torch.float32)[None]
    g = xs @ gate[..., :d].transpose(1, 2).contiguous()
    h = g * torch.sigmoid(g) * (xs @ up[..., :d].transpose(1, 2).contiguous())
    y = h @ down[..., :f].transpose(1, 2).contiguous()  # [experts][n][d]
    share = torch.zeros(n, state["experts"], device=x.device).scatter(1, ids, w)
    return (y * share.t()[..., None]).sum(0).to(torch.bfloat16)


# ---- the framework's calls --------------------------------------------------

def _handle24(a):
    import sparse_mask_search_amd as sms
    return sms.Sparse24Fp8(a["values"], a["meta"], a["scales"], a["k"])


def _own_quant(state):
    import sparse_mask_search_amd as sms
    x, out = state["x"], {}
    if state["along"] == "both":
        r, c = sms.quant_fp8_both(x)
        return {"rows": (r.values, r.scales), "cols": (c.values, c.scales)}
    q = sms.quant_fp8(x, transpose=state["along"] == "cols")
    return {state["along"]: (q.values, q.scales)}


def _own_compress(state):
    import sparse_mask_search_amd as sms
    if state["along"] == "both":
        r, c, bad, bad_t = sms.compress24_fp8_both(state["w"], state["mask"])
        return {"rows": (r.values, r.meta, r.scales, bad), "cols": (c.values, c.meta, c.scales, bad_t)}
    a, bad = sms.compress24_fp8(state["w"], state["mask"], transpose=state["along"] == "cols")
    return {state["along"]: (a.values, a.meta, a.scales, bad)}


def _own_linear(state):
    import sparse_mask_search_amd as sms
    return sms.spmm24_fp8(state["x"], _handle24(state["a"]))


def _own_wgrad(state):
    import sparse_mask_search_amd as sms
    return sms.gemm_fp8(sms.quant_fp8(state["dy"], transpose=True),
                        sms.quant_fp8(state["x"], transpose=True), mask=state["mask"])


def _own_moe(state):
    import sparse_mask_search_amd as sms
    return sms.moe24_fp8(state["x"], state["router"], _handle24(state["gate"]),
                         _handle24(state["up"]), _handle24(state["down"]), state["topk"])


def run(state):
    op = state["op"]
    if op == "quant":
        return _own_quant(state) if own else _plain_quant(state)
    if op == "compress":
        return _own_compress(state) if own else _plain_compress(state)
    if op == "linear":
        return _own_linear(state) if own else _plain_linear(state)
    if op == "wgrad":
        return _own_wgrad(state) if own else _plain_wgrad(state)
    return _own_moe(state) if own else _plain_moe(state)


# ---- what a pass cannot do without -------------------------------------------

def _bytes24(rows, k):
    return rows * k / 2 + rows * k / 8 + rows * k / 128 ** 2


def work(case):
    op = case["op"]
    if op == "quant":
        r, c = case["rows"], case["cols"]
        ways = 2 if case["along"] == "both" else 1
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": r * c * es + ways * (r * c + r * c / 128), "flops": ways * 2 * r * c}
    if op == "compress":
        r, c = case["rows"], case["cols"]
        ways = 2 if case["along"] == "both" else 1
        es = 2 if case["dtype"] == "bf16" else 4
        # only the kept half of the weights counts
        return {"bytes": r * c * es / 2 + r * c / 8 + ways * _bytes24(r, c), "flops": r * c}
    if op == "linear":
        n, m, k = case["n"], case["m"], case["k"]
        return {"bytes": n * k * 2 + _bytes24(m, k) + n * m * 2, "flops": n * m * k}
    if op == "wgrad":
        n, m, k = case["n"], case["m"], case["k"]
        return {"bytes": n * (m + k) * 2 + m * k / 8 + m * k * 2, "flops": n * m * k}
    n, d, f, e, topk = (case[c] for c in ("n", "d", "f", "experts", "topk"))
    hit = e * (1.0 - (1.0 - topk / e) ** n)  # experts that some token chose
    return {"bytes": n * d * 4 + e * d * 2 + hit * (2 * _bytes24(f, d) + _bytes24(d, f)),
            "flops": 2 * n * e * d + n * topk * 3 * d * f}


# ---- the definition in 64 bits, written apart from the plain form ---------------

def _ref_exponent(amax):
    s = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448.0))
    s = torch.where(amax > 448.0 * torch.exp2(s), s + 1, s)
    s = torch.where(amax <= 448.0 * torch.exp2(s - 1), s - 1, s).clamp(min=-127.0)
    return torch.where(amax == 0, torch.zeros_like(s), s)


def _ref_round(v):
    """Nearest e4m3 number, ties to even: 3 fraction bits, least exponent -6."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    e = torch.where(torch.exp2(e) > v.abs(), e - 1, e).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _ref_quant(x):
    r, c = x.shape
    full = torch.zeros(r, _up(c), dtype=torch.float64, device=x.device)
    full[:, :c] = x.to(torch.float64)
    s = _ref_exponent(full.abs().view(r, -1, 128).max(-1).values)
    wide = torch.exp2(s).repeat_interleave(128, 1)
    return _ref_round(full / wide), s, wide


def _ref_dense(a):
    v = a["values"].to(torch.float64)
    kp = v.shape[-1] * 2
    dense = torch.zeros(*v.shape[:-1], kp, dtype=torch.float64, device=v.device)
    slot = torch.arange(kp // 2, device=v.device)
    word = a["meta"].to(torch.int64)[..., slot // 16]
    pos = (word >> (2 * (slot % 16))) & 3
    dense.scatter_(-1, 4 * (slot // 2) + pos, v)
    s = torch.exp2(a["scales"].view(torch.uint8).to(torch.float64) - 127.0)
    r = torch.arange(v.shape[-2], device=v.device) // 128
    c = torch.arange(kp, device=v.device) // 128
    return dense * s[..., r[:, None], c[None, :]]


def _ref_compress(q, keep):
    """The kept entries of every group in order, by ranking the entries within their group."""
    r, kp = q.shape
    full = torch.zeros(r, kp, dtype=torch.bool, device=q.device)
    full[:, :keep.shape[1]] = keep
    k4 = full.view(r, -1, 4)
    rank = k4.cumsum(-1) - 1
    v = torch.zeros(r, kp // 4, 3, dtype=torch.float64, device=q.device)
    to = torch.where(k4 & (rank < 2), rank, torch.full_like(rank, 2))
    v.scatter_add_(-1, to, q.view(r, -1, 4))
    return v[..., :2].reshape(r, kp // 2)


def exact(case, seed):
    op = case["op"]
    state = prepare(case, seed)
    if op == "quant":
        out = {}
        if case["along"] in ("rows", "both"):
            q, s, _ = _ref_quant(state["x"])
            out["rows"] = (q, torch.exp2(s).t().contiguous())
        if case["along"] in ("cols", "both"):
            q, s, _ = _ref_quant(state["x"].t())
            out["cols"] = (q, torch.exp2(s).t().contiguous())
        return out
    if op == "compress":
        rows, cols = case["rows"], case["cols"]
        keep = _keep(state["mask"], cols)
        full = torch.zeros(_up(rows), _up(cols), dtype=torch.float64, device="cuda")
        full[:rows, :cols] = state["w"].to(torch.float64) * keep
        s = _ref_exponent(full.abs().view(-1, 128, _up(cols) // 128, 128).amax(3).amax(1))
        scale = torch.exp2(s)
        q = _ref_round(full / scale.repeat_interleave(128, 0).repeat_interleave(128, 1))
        out = {}
        if case["along"] in ("rows", "both"):
            out["rows"] = (_ref_compress(q[:rows], keep), None, scale, None)
        if case["along"] in ("cols", "both"):
            out["cols"] = (_ref_compress(q.t()[:cols].contiguous(), keep.t()), None, scale.t().contiguous(), None)
        return out
    if op == "linear":
        q, _, wide = _ref_quant(state["x"])
        return (q * wide) @ _ref_dense(state["a"]).t()
    if op == "wgrad":
        qy, _, wy = _ref_quant(state["dy"].t())
        qx, _, wx = _ref_quant(state["x"].t())
        return ((qy * wy) @ (qx * wx).t()) * _keep(state["mask"], case["k"])
    n, d, f = case["n"], case["d"], case["f"]
    x = state["x"].to(torch.float64)
    ids, w = _route(state["x"], state["router"], case["topk"], torch.float64)
    y = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.reshape(-1).tolist())):
        gate, up, down = (_ref_dense({c: state[p][c][e] for c in ("values", "meta", "scales")})
                          for p in ("gate", "up", "down"))
        t, j = (ids == e).nonzero(as_tuple=True)
        g = x[t] @ gate[:, :d].t()
        h = g / (1.0 + torch.exp(-g)) * (x[t] @ up[:, :d].t())
        y[t] += w[t, j][:, None] * (h @ down[:, :f].t())
    return y
