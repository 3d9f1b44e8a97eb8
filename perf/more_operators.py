"""Operators of expert layers and training steps of masked models, as cases to
measure: what each computes in elementary torch operations (the plain form), the
calls a user makes of this package for the same result, and the result from the
definition in 64 bits.

Rows sorted by expert: `ends` (int32, on the device) holds the row behind each
expert's last one, expert e owns rows ends[e - 1] .. ends[e] - 1 (from 0 for the
first).  Rows behind the last expert's belong to none; their results are zeros.

Operators (the "op" of a case):
  mm      products grouped by expert: Y = X W_e^T with W [experts][m][k]
          (forward), or Y = X W_e with W [experts][k][m] (data gradient), bf16
  wgrad   dW_e = dY_e^T X_e for every expert, kept where its mask keeps W
  quant   rows to 8-bit integers: scale amax / 127, nearest integer, ties to even
  int8    the product of 8-bit integers with a scale for each token and channel
          (tokens quantised on the way), for one weight or grouped by expert
  clip    the norm of all gradients of a model (of the entries that the masks
          keep) and the gradients scaled to at most a given norm
"""
import math
import random

import torch

own = False


def listed():
    return [
        # decoding: one token through many small experts
        {"name": "mm-6-of-64", "op": "mm", "rows": 6, "pad": 0, "experts": 64, "m": 1408, "k": 2048,
         "transpose": False},
        # a ragged serving batch, a few rows of the buffer unused
        {"name": "mm-1003-of-16", "op": "mm", "rows": 1003, "pad": 13, "experts": 16, "m": 2048, "k": 4096,
         "transpose": False},
        # a training step's forward through large experts
        {"name": "mm-16384-of-8", "op": "mm", "rows": 16384, "pad": 0, "experts": 8, "m": 11008, "k": 4096,
         "transpose": False},
        # a training step's data gradient
        {"name": "mm-8192-of-16-dgrad", "op": "mm", "rows": 8192, "pad": 0, "experts": 16, "m": 4096, "k": 2048,
         "transpose": True},
        # weight gradients of small experts from an odd number of tokens, fp32
        {"name": "wgrad-1001-of-4", "op": "wgrad", "rows": 1001, "pad": 0, "experts": 4, "m": 1024, "k": 1024,
         "dtype": "f32", "masked": False},
        # a training step's weight gradients under the experts' masks
        {"name": "wgrad-8192-of-16", "op": "wgrad", "rows": 8192, "pad": 0, "experts": 16, "m": 2048, "k": 4096,
         "dtype": "bf16", "masked": True},
        # a small fp32 layer
        {"name": "quant-1000x1028-f32", "op": "quant", "rows": 1000, "k": 1028, "dtype": "f32"},
        # an MLP projection's weights, or a long batch's activations
        {"name": "quant-11008x4096", "op": "quant", "rows": 11008, "k": 4096, "dtype": "bf16"},
        # decoding: one token through an attention projection
        {"name": "int8-1x4096x4096", "op": "int8", "rows": 1, "pad": 0, "experts": 0, "m": 4096, "k": 4096},
        # a long prompt through large experts
        {"name": "int8-8192-of-8", "op": "int8", "rows": 8192, "pad": 0, "experts": 8, "m": 11008, "k": 4096},
        # a small model's gradients: latency
        {"name": "clip-1x64-f32", "op": "clip", "layers": 1, "d": 64, "f": 172, "dtype": "f32", "masked": True},
        # four layers of a large model, projections under masks
        {"name": "clip-4x4096", "op": "clip", "layers": 4, "d": 4096, "f": 11008, "dtype": "bf16", "masked": True},
    ]


MOST_WEIGHTS = 8 * 11008 * 4096
MOST_PRODUCTS = 16384 * 11008 * 4096


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step))


def _sizes(rng, most_rows):
    """experts, m, k and rows of a grouped product within the largest listed one's cost."""
    step = rng.choice((1, 4, 8, 64))
    m, k = _log(rng, 128, 11008, step), _log(rng, 128, 11008, step)
    experts = rng.choice([e for e in (1, 4, 8, 16, 32, 64) if e * m * k <= MOST_WEIGHTS])
    rows = _log(rng, 1, most_rows)
    return experts, m, k, min(rows, MOST_PRODUCTS // (m * k))


def draw(rng):
    op = rng.choice(("mm", "mm", "wgrad", "quant", "int8", "int8", "clip"))
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 11008), "k": _log(rng, 32, 11008),
                "dtype": rng.choice(("bf16", "f32"))}
    if op == "clip":
        d = _log(rng, 64, 4096)
        return {"op": op, "layers": rng.randint(1, 4), "d": d, "f": _log(rng, d, 11008 * d // 4096),
                "dtype": rng.choice(("bf16", "f32")) if d <= 2048 else "bf16", "masked": rng.random() < 0.5}
    experts, m, k, rows = _sizes(rng, 8192 if op == "int8" else 16384)
    pad = rng.randint(0, rows // 8) if rng.random() < 0.3 else 0
    case = {"op": op, "rows": rows, "pad": pad, "experts": experts, "m": m, "k": k}
    if op == "mm":
        case["transpose"] = rng.random() < 0.4
    elif op == "wgrad":
        case["dtype"], case["masked"] = rng.choice(("bf16", "f32")), rng.random() < 0.5
    elif rng.random() < 0.5:
        case["experts"], case["pad"] = 0, 0  # one weight, no groups
    return case


def _up(v, q=128):
    return -(-v // q) * q


def _normal(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _words(gen, *shape):
    """Random mask words: half the entries kept."""
    return torch.randint(-2 ** 31, 2 ** 31, shape, device="cuda", generator=gen, dtype=torch.int64).to(torch.int32)


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _shapes(case):
    """The gradients of `layers` layers: four attention projections, three of the MLP, two norms."""
    d, f = case["d"], case["f"]
    return ([(d, d)] * 4 + [(f, d), (f, d), (d, f), (d,), (d,)]) * case["layers"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = dict(case)
    if op in ("mm", "wgrad", "int8"):
        rows, experts, m, k = (case[c] for c in ("rows", "experts", "m", "k"))
        if experts:
            # routing sends some experts two or three times as many rows as others
            rng = random.Random(seed)
            share = [math.exp(rng.gauss(0.0, 0.5)) for _ in range(experts)]
            counts = [0] * experts
            for e in rng.choices(range(experts), share, k=rows - case["pad"]):
                counts[e] += 1
            state["counts"] = counts
            state["ends"] = torch.tensor(counts, device="cuda").cumsum(0).to(torch.int32)
        if op == "wgrad":
            state["x"] = _normal(gen, rows, k).to(torch.bfloat16)
            state["dy"] = (1e-3 * _normal(gen, rows, m)).to(torch.bfloat16)
            state["mask"] = _words(gen, experts, m, _up(k, 32) // 32) if case["masked"] else None
        else:
            state["x"] = (_normal(gen, rows, k) * torch.exp(0.5 * _normal(gen, 1, k))).to(torch.bfloat16)
        lead = (experts,) if experts else ()
        if op == "mm":
            shape = (k, m) if case["transpose"] else (m, k)
            state["w"] = torch.stack([(0.02 * _normal(gen, *shape)).to(torch.bfloat16) for _ in range(experts)])
        elif op == "int8":
            # 0.02 * normal weights whose largest magnitude in a row is about 4 deviations
            w = torch.zeros(*lead, m, _up(k), device="cuda", dtype=torch.int8)
            for part in (w.unbind() if experts else (w,)):
                part[:, :k] = (32.0 * _normal(gen, m, k)).round_().clamp_(-127, 127)
            state["w"] = w
            state["ws"] = 0.02 / 32.0 * torch.exp(0.1 * _normal(gen, *lead, m))
    elif op == "quant":
        # activations with a few loud features
        x = _normal(gen, case["rows"], case["k"]) * torch.exp(_normal(gen, 1, case["k"]))
        state["x"] = x.to(_type(case))
    else:
        shapes = _shapes(case)
        size = 4.0 / math.sqrt(sum(math.prod(s) for s in shapes))  # a norm well above max_norm
        # projections in the case's type, norms in fp32 and without masks
        state["grads"] = [(size * _normal(gen, *s)).to(_type(case) if len(s) == 2 else torch.float32) for s in shapes]
        state["masks"] = [_words(gen, s[0], _up(s[1], 32) // 32) if len(s) == 2 else None for s in shapes] \
            if case["masked"] else None
        state["out"] = [torch.empty_like(g) for g in state["grads"]]
        state["max_norm"] = 1.0
    return state


# ---- plain form: fp32 throughout (64 bits where a sum is long or a value is next to a border) ----

def _keep(mask, cols):
    bits = (mask[..., None] >> torch.arange(32, device=mask.device, dtype=torch.int32)) & 1
    return bits.reshape(*mask.shape[:-1], -1)[..., :cols].bool()


def _parts(state, x):
    """The rows of each expert, then those that belong to none."""
    return x.split(state["counts"] + [state["pad"]])


def _plain_mm(state):
    def product(x, w):
        w = w.to(torch.float32)
        return x.to(torch.float32) @ (w if state["transpose"] else w.t())
    *parts, rest = _parts(state, state["x"])
    ys = [product(x, w).to(torch.bfloat16) for x, w in zip(parts, state["w"].unbind()) if x.shape[0]]
    return torch.cat(ys + [rest.new_zeros(rest.shape[0], state["m"])])


def _plain_wgrad(state):
    *xs, _ = _parts(state, state["x"])
    *dys, _ = _parts(state, state["dy"])
    masks = state["mask"].unbind() if state["masked"] else [None] * len(xs)

    def gradient(dy, x, mask):
        dw = dy.to(torch.float32).t() @ x.to(torch.float32)
        return (dw if mask is None else torch.where(_keep(mask, dw.shape[1]), dw, torch.zeros_like(dw))).to(_type(state))
    return torch.stack([gradient(dy, x, mask) for dy, x, mask in zip(dys, xs, masks)])


def _plain_quantised(x):
    """Integers [rows][kpad] as fp32, and scales: x * 127 / amax is taken in 64 bits, so that values
    next to a half go the right way."""
    wide = x.to(torch.float64)
    amax = wide.abs().amax(-1, keepdim=True)
    q = torch.where(amax > 0, (wide * 127.0) / amax, torch.zeros_like(wide)).round().to(torch.float32)
    return torch.nn.functional.pad(q, (0, _up(x.shape[1]) - x.shape[1])), (amax / 127.0).to(torch.float32)


def _plain_quant(state):
    q, s = _plain_quantised(state["x"])
    return q.to(torch.int8), s[:, 0]


def _plain_int8(state):
    q, s = _plain_quantised(state["x"])
    if not state["experts"]:
        return ((q @ state["w"].to(torch.float32).t()) * s * state["ws"]).to(torch.bfloat16)
    *qs, rest = _parts(state, q)
    *ss, _ = _parts(state, s)
    ys = [((x @ w.to(torch.float32).t()) * sx * sw).to(torch.bfloat16)
          for x, sx, w, sw in zip(qs, ss, state["w"].unbind(), state["ws"].unbind()) if x.shape[0]]
    return torch.cat(ys + [torch.zeros(rest.shape[0], state["m"], dtype=torch.bfloat16, device=q.device)])


def _plain_clip(state):
    masks = state["masks"] or [None] * len(state["grads"])
    kept = [g if m is None else torch.where(_keep(m, g.shape[1]), g, torch.zeros_like(g))
            for g, m in zip(state["grads"], masks)]
    norm = torch.stack([g.to(torch.float64).square().sum() for g in kept]).sum().sqrt()
    factor = (state["max_norm"] / norm).clamp(max=1.0).to(torch.float32)
    return norm.to(torch.float32), [(g.to(torch.float32) * factor).to(g.dtype) for g in kept]


# ---- the framework's calls --------------------------------------------------

def _own_mm(state):
    import sparse_mask_search_amd as sms
    return sms.grouped_mm(state["x"], state["w"], state["ends"], transpose=state["transpose"])


def _own_wgrad(state):
    import sparse_mask_search_amd as sms
    return sms.grouped_wgrad(state["dy"], state["x"], state["ends"], mask=state["mask"], dtype=_type(state))


def _own_quant(state):
    import sparse_mask_search_amd as sms
    q = sms.quant_int8(state["x"])
    return q.values, q.scales


def _own_int8(state):
    import sparse_mask_search_amd as sms
    a = sms.DenseInt8(state["w"], state["ws"], state["k"])
    return sms.gemm_int8(state["x"], a, ends=state["ends"]) if state["experts"] else sms.gemm_int8(state["x"], a)


def _own_clip(state):
    import sparse_mask_search_amd as sms
    norm = sms.clip_grads(state["grads"], state["max_norm"], masks=state["masks"], out=state["out"])
    return norm, state["out"]


def run(state):
    op = state["op"]
    if op == "mm":
        return _own_mm(state) if own else _plain_mm(state)
    if op == "wgrad":
        return _own_wgrad(state) if own else _plain_wgrad(state)
    if op == "quant":
        return _own_quant(state) if own else _plain_quant(state)
    if op == "int8":
        return _own_int8(state) if own else _plain_int8(state)
    return _own_clip(state) if own else _plain_clip(state)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    op = case["op"]
    if op == "quant":
        r, k = case["rows"], case["k"]
        return {"bytes": r * k * (2 if case["dtype"] == "bf16" else 4) + r * _up(k) + 4 * r, "flops": 2 * r * k}
    if op == "clip":
        size = 0
        for s in _shapes(case):
            n = math.prod(s)
            size += 2 * n * (2 if case["dtype"] == "bf16" and len(s) == 2 else 4)
            size += n / 8 if case["masked"] and len(s) == 2 else 0
        return {"bytes": size, "flops": 3 * sum(math.prod(s) for s in _shapes(case))}
    rows, experts, m, k = (case[c] for c in ("rows", "experts", "m", "k"))
    n = rows - case["pad"]
    hit = experts * (1.0 - (1.0 - 1.0 / experts) ** n) if experts else 1  # experts that some row went to
    flops = 2 * n * m * k
    if op == "mm":
        return {"bytes": 2 * (n * k + hit * m * k + rows * m), "flops": flops}
    if op == "wgrad":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * (m + k) + experts * m * k * (es + (1 / 8 if case["masked"] else 0)), "flops": flops}
    return {"bytes": 2 * n * k + hit * m * (k + 4) + 2 * rows * m, "flops": flops}


# ---- the definition in 64 bits, written apart from the plain form ---------------

def _ref_round(v):
    """Nearest integer, ties to the even one."""
    low = torch.floor(v)
    over = v - low
    return low + (over > 0.5) + ((over == 0.5) & (torch.remainder(low, 2.0) == 1.0))


def _ref_bits(mask, cols):
    c = torch.arange(cols, device=mask.device)
    return ((mask.to(torch.int64)[..., c // 32] >> (c % 32)) % 2).to(torch.float64)


def _ref_rows(state):
    """(expert, first row, last row + 1) of every expert."""
    ends = state["ends"].tolist()
    return [(e, ends[e - 1] if e else 0, ends[e]) for e in range(len(ends))]


def exact(case, seed):
    op = case["op"]
    state = prepare(case, seed)
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        kept = []
        for i, g in enumerate(state["grads"]):
            v = g.to(torch.float64)
            if state["masks"] is not None and state["masks"][i] is not None:
                v = v * _ref_bits(state["masks"][i], g.shape[1])
            total = total + (v * v).sum()
            kept.append(g if case["d"] > 1024 else v)
        norm = torch.sqrt(total)
        if case["d"] > 1024:
            return norm, [None] * len(kept)
        return norm, [v * (state["max_norm"] / norm) if norm > state["max_norm"] else v for v in kept]
    if op == "quant":
        s = state["x"].to(torch.float64).abs().max(-1).values / 127.0
        return None, s
    x = state["x"].to(torch.float64)
    if op == "wgrad":
        dy = state["dy"].to(torch.float64)
        out = torch.empty(case["experts"], case["m"], case["k"], dtype=torch.float64, device="cuda")
        for e, first, end in _ref_rows(state):
            out[e] = dy[first:end].t() @ x[first:end]
            if case["masked"]:
                out[e] *= _ref_bits(state["mask"][e], case["k"])
        return out
    y = torch.zeros(case["rows"], case["m"], dtype=torch.float64, device="cuda")
    if op == "mm":
        for e, first, end in _ref_rows(state):
            w = state["w"][e].to(torch.float64)
            y[first:end] = x[first:end] @ (w if case["transpose"] else w.t())
        return y
    amax = x.abs().max(-1, keepdim=True).values
    x = _ref_round(x * 127.0 / amax.clamp(min=1e-300)) * (amax / 127.0)
    k = case["k"]
    if not case["experts"]:
        return x @ (state["w"][:, :k].to(torch.float64) * state["ws"].to(torch.float64)[:, None]).t()
    for e, first, end in _ref_rows(state):
        y[first:end] = x[first:end] @ (state["w"][e, :, :k].to(torch.float64) * state["ws"][e].to(torch.float64)[:, None]).t()
    return y
