"""GPU: the dense operators of masked models (include/tsenor_ops.h) against numpy in 64 bits:
bit for bit where every number is a small integer (products and sums are exact then, and only
the output type rounds), and within the bounds below otherwise.

Bounds.  Products of bf16 numbers are exact in fp32.  A sum of k of them has k additions; each is off by
at most 2^-23 of a partial sum (the matrix cores may cut where IEEE rounds), which the sum of magnitudes
bounds.  The output type rounds last, by half a step (2^-8 relative in bf16, 2^-24 in fp32).
"""
import numpy as np
import pytest

import ops_ref as ref
import sparse_mask_search_amd as sms
from sparse_mask_search_amd import workloads as wl
from gpu_util import to_device

pytestmark = pytest.mark.gpu


def say(*a):
    print("[case]", *a, flush=True)


def f64(t):
    import torch
    torch.cuda.synchronize()
    return t.to(torch.float32).cpu().numpy().astype(np.float64)


def bf16(x):
    """A device tensor of fp64 values and the values it holds."""
    x = np.asarray(x, np.float32)
    bits = wl.f32_to_bf16_bits(x.reshape(1, -1)).reshape(x.shape)
    held = wl.bf16_bits_to_f32(bits.reshape(1, -1)).reshape(x.shape).astype(np.float64)
    return to_device(bits), held


def ints(rng, shape, most=3):
    return rng.integers(-most, most + 1, shape).astype(np.float64)


def ends_of(counts):
    import torch
    return torch.tensor(np.cumsum(counts), dtype=torch.int32).cuda()


def words(keep):
    import torch
    return torch.from_numpy(ref.pack_mask(keep).view(np.int32)).cuda()


def torch_type(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def exactly(got, want):
    """Equal to the fp64 values rounded to got's type."""
    import torch
    want = torch.from_numpy(np.asarray(want, np.float32)).to(got.dtype).to(torch.float64).numpy()
    g = f64(got)
    assert g.shape == want.shape
    same = (g == want) | (np.isnan(g) & np.isnan(want))
    assert same.all(), (int((~same).sum()), np.argwhere(~same)[:4].tolist())


def close(got, want, absum, k):
    import torch
    slack = k * 2.0 ** -23 * absum
    tol = slack + torch.finfo(got.dtype).eps / 2 * (np.abs(want) + slack) + 1e-38
    err = np.abs(f64(got) - want)
    assert got.shape == want.shape and (err <= tol).all(), (float(err.max()), float((err / tol).max()))


COUNTS = [
    ([1], 0), ([7], 0), ([0, 5, 0, 70, 1], 3), ([0, 0, 0], 2), ([64, 128, 63], 0), ([33, 0, 300, 17], 5),
    ([1, 0, 2] * 60, 1), ([0] * 70 + [9] + [0] * 70, 0),
]
SIZES = [(1, 1), (64, 32), (100, 72), (257, 131), (48, 1000), (384, 520)]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("m,k", SIZES)
@pytest.mark.parametrize("counts,pad", COUNTS, ids=lambda v: "" if isinstance(v, int) else f"{len(v)}x{sum(v)}")
def test_grouped_mm_exact(counts, pad, m, k, transpose):
    say("grouped_mm", len(counts), sum(counts), pad, m, k, transpose)
    rng = np.random.default_rng(m + k + len(counts))
    x, xv = bf16(ints(rng, (sum(counts) + pad, k)))
    w, wv = bf16(ints(rng, (len(counts), k, m) if transpose else (len(counts), m, k)))
    want, _ = ref.grouped_mm(xv, wv, np.cumsum(counts), transpose)
    for name in ("bf16", "f32"):
        exactly(sms.grouped_mm(x, w, ends_of(counts), transpose=transpose, dtype=torch_type(name)), want)


@pytest.mark.parametrize("dtype,masked", [("bf16", True), ("f32", False), ("f32", True), ("bf16", False)])
@pytest.mark.parametrize("m,k", SIZES)
@pytest.mark.parametrize("counts,pad", COUNTS[:6], ids=lambda v: "" if isinstance(v, int) else f"{len(v)}x{sum(v)}")
def test_grouped_wgrad_exact(counts, pad, m, k, dtype, masked):
    say("grouped_wgrad", len(counts), sum(counts), pad, m, k, dtype, masked)
    rng = np.random.default_rng(m * 3 + k + len(counts))
    x, xv = bf16(ints(rng, (sum(counts) + pad, k)))
    dy, dyv = bf16(ints(rng, (sum(counts) + pad, m)))
    keep = rng.random((len(counts), m, k)) < 0.5 if masked else None
    want, _ = ref.grouped_wgrad(dyv, xv, np.cumsum(counts), keep)
    exactly(sms.grouped_wgrad(dy, x, ends_of(counts), mask=words(keep) if masked else None,
                              dtype=torch_type(dtype)), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped_rounding(dtype):
    """Real numbers, long reductions: within the bound of the sums."""
    rng = np.random.default_rng(5)
    counts = [100, 3, 0, 700]
    x, xv = bf16(rng.standard_normal((803, 1200)))
    w, wv = bf16(rng.standard_normal((4, 130, 1200)))
    dy, dyv = bf16(rng.standard_normal((803, 130)))
    t = torch_type(dtype)
    want, s = ref.grouped_mm(xv, wv, np.cumsum(counts), False)
    close(sms.grouped_mm(x, w, ends_of(counts), dtype=t), want, s, 1200)
    want, s = ref.grouped_mm(dyv, wv, np.cumsum(counts), True)
    close(sms.grouped_mm(dy, w, ends_of(counts), transpose=True, dtype=t), want, s, 130)
    want, s = ref.grouped_wgrad(dyv, xv, np.cumsum(counts))
    close(sms.grouped_wgrad(dy, x, ends_of(counts), dtype=t), want, s, 700)


HARD = [0.0, 1.0, -1.0, 0.5, 63.5 / 127, -2.5 / 127, 1.5 / 127, 1e-3]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 500), (5, 128), (130, 131), (9, 2049), (33, 4096), (3, 5000), (2, 20000)])
def test_quant_int8_exact(rows, k, dtype):
    """Ties (entries that are odd multiples of amax / 254), subnormals, large numbers, rows of zeros,
    rows with an infinity or a NaN."""
    import torch
    say("quant_int8", rows, k, dtype)
    rng = np.random.default_rng(rows * k)
    x = rng.standard_normal((rows, k)).astype(np.float32)
    x[::2] *= np.float32(127.0) / np.abs(x[::2]).max(-1, keepdims=True)
    x[::2] = np.rint(x[::2] * 2) / 2  # many exact halves: amax is 127
    if rows > 1:
        x[1] = 2.0 ** rng.integers(-9, 1, k) * rng.choice([-1, 1], k)  # amax / 2 is a tie, 63.5
    if rows > 4:
        x[2], x[3], x[4] = 0.0, x[3] * np.float32(1e-41), x[4] * np.float32(1e37)
    if rows > 8:
        x[5, k // 2], x[7, 0], x[8] = np.inf, np.nan, x[8] * np.float32(1e-38)
    t = torch.from_numpy(x).cuda().to(torch_type(dtype))
    held = t.to(torch.float32).cpu().numpy()
    q = sms.quant_int8(t)
    values, scales = ref.quant_int8(held)
    assert q.k == k and np.array_equal(q.values.cpu().numpy(), values)
    assert np.array_equal(q.scales.cpu().numpy(), scales, equal_nan=True)


def test_quant_int8_every_bf16_pair():
    """Every bf16 magnitude within 2^-9 of amax against amax of every significand."""
    import torch
    m = np.arange(128, 256)
    x = np.concatenate([(m / 2.0 ** s) for s in range(0, 10)])[None, :].repeat(128, 0)
    x = np.where(x > m[:, None], 0.0, x)
    x = np.concatenate([x, m[:, None].astype(float)], 1).astype(np.float32)
    q = sms.quant_int8(torch.from_numpy(x).cuda().to(torch.bfloat16))
    assert np.array_equal(q.values.cpu().numpy(), ref.quant_int8(x)[0])


def _int8_operands(rng, lead, rows, k):
    import torch
    v = np.zeros((*lead, rows, ref.pad(k)), np.int8)
    v[..., :k] = rng.integers(-127, 128, (*lead, rows, k))
    s = (2.0 ** rng.integers(-8, 3, (*lead, rows)) * rng.uniform(0.5, 1, (*lead, rows))).astype(np.float32)
    return v, s, sms.DenseInt8(torch.from_numpy(v).cuda(), torch.from_numpy(s).cuda(), k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,m,k", [(1, 1, 1), (1, 100, 500), (16, 64, 128), (17, 130, 1000), (70, 257, 300),
                                      (300, 384, 2048), (3, 40, 131072)])
def test_gemm_int8_exact(rows, m, k, dtype):
    say("gemm_int8", rows, m, k, dtype)
    rng = np.random.default_rng(rows + m)
    xv, xs, x = _int8_operands(rng, (), rows, k)
    av, as_, a = _int8_operands(rng, (), m, k)
    exactly(sms.gemm_int8(x, a, dtype=torch_type(dtype)), ref.gemm_int8(xv, xs, av, as_))


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 100])
@pytest.mark.parametrize("k", [1, 136, 1000, 4096])
@pytest.mark.parametrize("xtype", ["bf16", "f32"])
def test_gemm_int8_quantises(rows, k, xtype):
    """Tokens given as they are: the same as from quant_int8."""
    import torch
    rng = np.random.default_rng(rows + k)
    x = torch.from_numpy(rng.standard_normal((rows, k)).astype(np.float32)).cuda().to(torch_type(xtype))
    if rows > 2:
        x[1] = 0
        x[2, k // 2] = float("nan")
    _, _, a = _int8_operands(rng, (), 77, k)
    q = sms.quant_int8(x)
    want = ref.gemm_int8(q.values.cpu().numpy(), q.scales.cpu().numpy(), a.values.cpu().numpy(), a.scales.cpu().numpy())
    exactly(sms.gemm_int8(x, a, dtype=torch.float32), want)


@pytest.mark.parametrize("counts,pad", COUNTS, ids=lambda v: "" if isinstance(v, int) else f"{len(v)}x{sum(v)}")
def test_gemm_int8_grouped(counts, pad):
    import torch
    rng = np.random.default_rng(len(counts))
    rows, m, k = sum(counts) + pad, 150, 200
    xv, xs, x = _int8_operands(rng, (), rows, k)
    av, as_, a = _int8_operands(rng, (len(counts),), m, k)
    want = np.zeros((rows, m), np.float32)
    for e, (i, j) in enumerate(ref.bounds(np.cumsum(counts), rows)):
        want[i:j] = ref.gemm_int8(xv[i:j], xs[i:j], av[e], as_[e])
    exactly(sms.gemm_int8(x, a, ends=ends_of(counts), dtype=torch.float32), want)


def _clip_check(grads, got, keeps, max_norm, norm):
    """norm: the sum of squares in 64 bits, off by 2^-53 an addition, rounded to fp32.  The factor is
    off by one fp32 rounding; the product rounds once to the gradient's type."""
    import torch
    vals = [f64(g) * (1.0 if k is None else k) for g, k in zip(grads, keeps)]
    want = np.sqrt(sum(float((v * v).sum()) for v in vals))
    assert abs(float(norm) - want) <= want * (2.0 ** -24 + 1e-9)
    f = min(1.0, max_norm / want) if want > 0 else 1.0
    for v, g in zip(vals, got):
        tol = np.abs(v * f) * (torch.finfo(g.dtype).eps / 2 * (1 + 2.0 ** -23) + 2.0 ** -23) + 2.0 ** -134
        assert (np.abs(f64(g) - v * f) <= (tol if f < 1.0 else 0.0)).all()


@pytest.mark.parametrize("max_norm", [0.5, 1e6, 0.0])
@pytest.mark.parametrize("count", [1, 9, 100])
@pytest.mark.parametrize("masked", [False, True])
def test_clip_grads(count, masked, max_norm):
    import torch
    rng = np.random.default_rng(count)
    shapes = [(8, 64), (3, 5), (1000,), (), (7, 33), (2, 3, 40), (260, 519), (64, 1024), (1, 1), (0, 5)]
    grads, keeps, masks = [], [], []
    for i in range(count):
        s = shapes[i % len(shapes)]
        g = torch.tensor(np.asarray(rng.standard_normal(s)) * 0.1, dtype=torch.float32).cuda()
        grads.append(g.to(torch.bfloat16) if i % 3 else g)
        keep = rng.random(s) < 0.5 if masked and len(s) > 1 and i % 4 else None
        keeps.append(keep)
        masks.append(None if keep is None else words(keep))
    before = [g.clone() for g in grads]
    norm = sms.grad_norm(grads, masks=masks)
    out = [torch.full_like(g, 7.0) for g in grads]
    norm2 = sms.clip_grads(grads, max_norm, masks=masks, out=out)
    assert float(norm) == float(norm2) and all(torch.equal(a, b) for a, b in zip(before, grads))
    _clip_check(before, out, keeps, max_norm, norm)
    norm3 = sms.clip_grads(grads, max_norm, masks=masks)
    assert float(norm3) == float(norm) and all(torch.equal(a, b) for a, b in zip(out, grads))


def test_training_step_of_a_masked_expert_layer():
    """mask -> forward -> data gradient -> masked weight gradient -> clipping, and the 8-bit integer
    form of the same layer.  All numbers are integers, so gradients equal differences exactly."""
    import torch
    rng = np.random.default_rng(11)
    counts, m, k = [40, 0, 130, 9], 128, 96
    rows, ends = sum(counts) + 4, ends_of(counts)
    w = torch.from_numpy(ints(rng, (4, m, k), 2).astype(np.float32)).cuda().to(torch.bfloat16)
    mask = torch.stack([sms.mask(w[e].contiguous(), 8, 16, 20.0, 40, 8)[0] for e in range(4)])
    keep = torch.stack([sms.unpack(mask[e], k) for e in range(4)])
    w = w * keep
    x, xv = bf16(ints(rng, (rows, k), 2))
    dy, dyv = bf16(ints(rng, (rows, m), 2))
    f32 = torch.float32
    y = sms.grouped_mm(x, w, ends, dtype=f32)
    dx = sms.grouped_mm(dy, w, ends, transpose=True, dtype=f32)
    dw = sms.grouped_wgrad(dy, x, ends, mask=mask, dtype=f32)
    wv, kv = f64(w), keep.cpu().numpy()
    exactly(y, ref.grouped_mm(xv, wv, np.cumsum(counts), False)[0])
    exactly(dx, ref.grouped_mm(dyv, wv, np.cumsum(counts), True)[0])
    exactly(dw, ref.grouped_wgrad(dyv, xv, np.cumsum(counts), kv)[0])

    def loss(w_, x_):
        return float((f64(sms.grouped_mm(x_, w_, ends, dtype=f32)) * dyv).sum())
    base = loss(w, x)
    for e, i, j in [(0, 3, 5), (2, 127, 95), (2, 64, 0), (3, 1, 1), (1, 2, 2)]:
        w2 = w.clone()
        w2[e, i, j] += 1
        change = loss(w2, x) - base
        assert float(dw[e, i, j]) == (change if kv[e, i, j] else 0.0)
    for r, j in [(0, 0), (39, 95), (100, 17), (rows - 1, 3)]:
        x2 = x.clone()
        x2[r, j] += 1
        assert float(dx[r, j]) == loss(w, x2) - base
    before = [dw.clone(), dx.clone()]
    norm = sms.clip_grads([dw, dx], 1.0, masks=[mask, None])
    _clip_check(before, [dw, dx], [kv, None], 1.0, norm)
    # serving: the weights' integers stand for them, up to half a step of each row's scale
    a = sms.quant_int8(w)
    q = sms.quant_int8(x)
    y8 = f64(sms.gemm_int8(x, a, ends=ends, dtype=f32))
    wq = a.values.cpu().numpy()[..., :k].astype(np.float64) * a.scales.cpu().numpy()[..., None].astype(np.float64)
    xq = q.values.cpu().numpy()[:, :k].astype(np.float64) * q.scales.cpu().numpy()[:, None].astype(np.float64)
    assert (np.abs(wq - wv) <= np.abs(wv).max(-1, keepdims=True) / 254 * (1 + 2.0 ** -20)).all()
    want, s = ref.grouped_mm(xq, wq, np.cumsum(counts), False)
    assert (np.abs(y8 - want) <= 3 * 2.0 ** -23 * s + 1e-30).all()
