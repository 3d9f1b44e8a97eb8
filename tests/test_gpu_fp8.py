"""GPU: the 8-bit operators of 2:4-masked weights (include/tsenor_fp8.h) against
numpy in 64 bits: operands bit for bit; products bit for bit where every
number is a small integer times a power of two (nothing is rounded before the
output type then), and within the bounds below otherwise.

Bounds.  The 8-bit matrix cores add eight products at a time and cut each 2^-12
below the largest of the eight or lower (measured: addends at 2^-12 are whole,
at 2^-14 gone), so a sum loses at most 7 * 2^-12 of the sum of magnitudes.  What
follows is fp32: one rounding (2^-24 of a partial sum, at most the sum of
magnitudes) for each group of eight, each scaling and each block.  The output
type rounds last, by half a step (2^-8 relative in bf16, 2^-24 in fp32).
"""
import numpy as np
import pytest

import fp8_ref as ref
import oracle
import sparse_mask_search_amd as sms
from sparse_mask_search_amd import workloads as wl
from gpu_util import to_device

pytestmark = pytest.mark.gpu

CUT = 7 * 2.0 ** -12


def say(*a):
    print("[case]", *a, flush=True)


def sync():
    import torch
    torch.cuda.synchronize()


def bytes_of(t):
    import torch
    return t.contiguous().view(torch.uint8).cpu().numpy()


def f64(t):
    import torch
    return t.to(torch.float32).cpu().numpy().astype(np.float64)


def tensor(x, dtype):
    """A device tensor of fp64 values and the values it holds."""
    x32 = np.asarray(x, np.float32)
    if dtype == "bf16":
        bits = wl.f32_to_bf16_bits(x32)
        return to_device(bits), wl.bf16_bits_to_f32(bits).astype(np.float64)
    return to_device(x32), x32.astype(np.float64)


def words(keep):
    import torch
    return torch.from_numpy(ref.pack_mask(keep).view(np.int32)).cuda()


def half_step(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


def close(got, want, absum, rel, dtype):
    """|got - want| <= rel * absum, then the rounding to dtype (of a value that is off by that)."""
    slack = rel * absum
    tol = slack + half_step(dtype) * (np.abs(want) + slack) + 1e-38
    err = np.abs(f64(got) - want)
    assert got.shape == want.shape and np.isfinite(f64(got)).all()
    assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))


def sum_rel(k):
    """Bound of a sum along k, relative to the sum of magnitudes."""
    return CUT + (2 * -(-k // 8) + 2) * 2.0 ** -24


def powers(rng, rows, cols, most=3):
    """Powers of two, one for each 1 x 128 block, as a factor for integer entries."""
    return np.repeat(2.0 ** rng.integers(-most, most + 1, (rows, -(-cols // 128))), 128, 1)[:, :cols]


def powers_square(rng, rows, cols, most=3):
    return np.repeat(powers(rng, -(-rows // 128), cols, most), 128, 0)[:rows]


def integers(rng, shape, most):
    return rng.integers(-most, most + 1, shape).astype(np.float64)


# ---- quantisation -----------------------------------------------------------

def _hard_values(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * np.exp(2 * rng.standard_normal((1, cols)))
    x[rng.random((rows, cols)) < 0.05] = 0.0
    x[::3] *= 2.0 ** -40
    if rows > 2:
        x[1] = 0.0
        x[2, :: 7] = 448.0 * 2.0 ** 3   # exactly on the border of a scale
    if rows > 4:
        x[4] = 1e-38 * rng.standard_normal(cols)   # subnormals, the clamp of the scale
        x[3] = 3e38 * rng.uniform(-1, 1, cols)
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 500), (5, 128), (130, 131), (300, 264), (64, 1024)])
def test_quant_bit_exact(rows, cols, dtype):
    say("quant", rows, cols, dtype)
    x, xv = tensor(_hard_values(np.random.default_rng(rows + cols), rows, cols), dtype)
    a, t = sms.quant_fp8(x), sms.quant_fp8(x, transpose=True)
    a2, t2 = sms.quant_fp8_both(x)
    sync()
    for op, v in ((a, xv), (t, xv.T), (a2, xv), (t2, xv.T)):
        codes, scales, _ = ref.quant(v)
        assert op.k == v.shape[1]
        assert np.array_equal(bytes_of(op.scales), scales)
        got = bytes_of(op.values)
        assert np.array_equal(got, codes), np.argwhere(got != codes)[:5]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quant_non_finite_and_strides(dtype):
    import torch
    rng = np.random.default_rng(5)
    x = rng.standard_normal((140, 300))
    x[0, 3], x[7, 130], x[20, 299] = np.inf, -np.inf, np.nan
    x[9] = np.inf
    big, _ = tensor(rng.standard_normal((150, 333)), dtype)
    part = big[5:145, 7:307]             # rows that are not 16-byte aligned
    part.copy_(tensor(x, dtype)[0])
    xv = tensor(x, dtype)[1]
    for op, v in zip(sms.quant_fp8_both(part), (xv, xv.T)):
        sync()
        codes, scales, _ = ref.quant(v)
        got = bytes_of(op.values)
        nan = (codes & 0x7F) == 0x7F
        assert np.array_equal(bytes_of(op.scales), scales)
        assert np.array_equal((got & 0x7F) == 0x7F, nan) and np.array_equal(got[~nan], codes[~nan])
    assert torch.equal(sms.quant_fp8(part[:1]).values.view(torch.uint8),
                       sms.quant_fp8(part).values.view(torch.uint8)[:1])


def test_quant_no_rows():
    import torch
    x = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda")
    a, t = sms.quant_fp8_both(x)
    assert a.values.shape == (0, 128) and a.scales.shape == (1, 0)
    assert t.values.shape == (40, 0) and t.scales.shape == (0, 40) and t.k == 0


# ---- compression ------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(4, 4), (36, 60), (132, 260), (256, 128)])
def test_compress_bit_exact(rows, cols, dtype):
    say("compress", rows, cols, dtype)
    rng = np.random.default_rng(rows * cols)
    w, wv = tensor(0.02 * rng.standard_normal((rows, cols)), dtype)
    keep = ref.random24(rng, rows, cols)
    m = words(keep)
    one, bad1 = sms.compress24_fp8(w, m)
    two, bad2 = sms.compress24_fp8(w, m, transpose=True)
    a, t, bad, bad_t = sms.compress24_fp8_both(w, m)
    sync()
    assert [int(b.item()) for b in (bad1, bad2, bad, bad_t)] == [0, 0, 0, 0]
    dense = []
    for op, v, kp in ((one, wv, keep), (a, wv, keep), (two, wv.T, keep.T), (t, wv.T, keep.T)):
        codes, meta, scales, _, d = ref.compress(v, kp)
        assert np.array_equal(bytes_of(op.values), codes)
        assert np.array_equal(op.meta.cpu().numpy().view(np.uint32), meta)
        assert np.array_equal(bytes_of(op.scales), scales)
        dense.append(d)
    assert np.array_equal(dense[1][:, :cols], dense[3][:, :rows].T)  # the same 8-bit numbers


def test_compress_any_mask_stack_and_strides():
    """A stack of matrices in a wider buffer, a mask that is not 2:4 (groups with
    more than two kept entries are counted, groups with none are empty), bits
    behind the last column set."""
    import torch
    rng = np.random.default_rng(3)
    e, rows, cols = 3, 36, 140
    keep = rng.random((e, rows, cols)) < 0.45
    keep[1] = False
    buf, _ = tensor(rng.standard_normal((e * (rows + 1), cols + 9)), "f32")
    w = buf.view(e, rows + 1, cols + 9)[:, :rows, 1:cols + 1]
    wv = w.cpu().numpy().astype(np.float64)
    mw = np.stack([ref.pack_mask(k) for k in keep])
    mw[..., -1] |= np.uint32(0xFFFFFFFF << (cols % 32) & 0xFFFFFFFF)
    a, t, bad, bad_t = sms.compress24_fp8_both(w, torch.from_numpy(mw.view(np.int32)).cuda())
    sync()
    for op, count, turn in ((a, bad, False), (t, bad_t, True)):
        total = 0
        for i in range(e):
            v, kp = (wv[i].T, keep[i].T) if turn else (wv[i], keep[i])
            codes, meta, scales, b, _ = ref.compress(v, kp)
            total += b
            assert np.array_equal(bytes_of(op.values[i]), codes)
            assert np.array_equal(op.meta[i].cpu().numpy().view(np.uint32), meta)
            assert np.array_equal(bytes_of(op.scales[i]), scales)
        assert int(count.item()) == total > 0


# ---- the product with a 2:4 operand ------------------------------------------

def _weight(rng, m, k, dtype="bf16"):
    w, wv = tensor(0.05 * rng.standard_normal((m, k)) * np.exp(0.7 * rng.standard_normal((m, 1))), dtype)
    keep = ref.random24(rng, m, k)
    return w, wv, keep


SHAPES = [(4, 4), (16, 128), (100, 132), (260, 516), (128, 1024), (512, 256), (96, 60)]


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("n", [1, 3, 16, 17, 40, 64, 65, 130, 257])
def test_spmm(n, m, k):
    import torch
    say("spmm", n, m, k)
    rng = np.random.default_rng(n + m + k)
    w, wv, keep = _weight(rng, m, k)
    A, _ = sms.compress24_fp8(w, words(keep))
    dense = ref.compress(wv, keep)[4]
    x, xv = tensor(rng.standard_normal((n, k)) * np.exp(rng.standard_normal((1, k))), "bf16")
    xd = ref.quant(xv)[2]
    want, absum = xd @ dense.T, np.abs(xd) @ np.abs(dense).T
    for dt in (torch.bfloat16, torch.float32):
        for X in (x, sms.quant_fp8(x)):
            y = sms.spmm24_fp8(X, A, dtype=dt)
            sync()
            assert y.dtype == dt
            close(y, want, absum, sum_rel(k), dt)


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("n", [1, 3, 16, 17, 40, 64, 65, 130, 257, 520])
def test_spmm_exact(n, m, k):
    """Integers up to 7, scaled by a power of two for each block: sums are exact in fp32."""
    import torch
    say("spmm exact", n, m, k)
    rng = np.random.default_rng(n * m + k)
    keep = ref.random24(rng, m, k)
    w, wv = tensor(integers(rng, (m, k), 7) * powers_square(rng, m, k), "bf16")
    x, xv = tensor(integers(rng, (n, k), 7) * powers(rng, n, k), "bf16")
    A, _ = sms.compress24_fp8(w, words(keep))
    want = xv @ np.where(keep, wv, 0).T
    for X in (x, sms.quant_fp8(x), x.float()):
        y, yb = sms.spmm24_fp8(X, A, dtype=torch.float32), sms.spmm24_fp8(X, A)
        sync()
        assert np.array_equal(f64(y), want)
        assert torch.equal(yb, y.bfloat16())


def test_spmm_f32_activations_and_transposed_operand():
    """The data gradient: dX = dY W with the operand of W^T."""
    import torch
    rng = np.random.default_rng(8)
    m, k, n = 260, 132, 50
    w, wv, keep = _weight(rng, m, k)
    T, _ = sms.compress24_fp8(w, words(keep), transpose=True)
    dense = ref.compress(wv, keep)[4][:, :k]
    dy, dyv = tensor(1e-4 * rng.standard_normal((n, m)), "f32")
    g = ref.quant(dyv)[2][:, :m]
    dx = sms.spmm24_fp8(dy, T, dtype=torch.float32)
    sync()
    close(dx, g @ dense, np.abs(g) @ np.abs(dense), sum_rel(m), torch.float32)


@pytest.mark.parametrize("n", [2, 16, 70, 300])
def test_spmm_writes_its_part_only(n):
    """Strided X and Y, sizes that end inside every tile: what lies around Y stays."""
    import torch
    rng = np.random.default_rng(n)
    m, k = 132, 388
    w, wv, keep = _weight(rng, m, k)
    A, _ = sms.compress24_fp8(w, words(keep))
    dense = ref.compress(wv, keep)[4]
    wide, _ = tensor(rng.standard_normal((n, k + 13)), "bf16")
    x = wide[:, 5:5 + k]
    xd = ref.quant(f64(x))[2]
    for dt, off in ((torch.bfloat16, 3), (torch.float32, 4)):
        buf = torch.full((n + 4, m + 12), 7.0, dtype=dt, device="cuda")
        y = buf[2:2 + n, off:off + m]
        assert sms.spmm24_fp8(x, A, out=y) is y
        sync()
        close(y, xd @ dense.T, np.abs(xd) @ np.abs(dense).T, sum_rel(k), dt)
        y.fill_(7.0)
        assert bool((buf == 7.0).all())


@pytest.mark.parametrize("n", [3, 40, 300])
def test_spmm_nan_stays_in_its_row_and_extreme_scales(n):
    import torch
    rng = np.random.default_rng(2)
    m, k = 64, 256
    w, wv, keep = _weight(rng, m, k)
    keep[0] = False                       # a row of A without entries
    wv = wv * 2.0 ** -60
    w = w * 2.0 ** -60
    A, _ = sms.compress24_fp8(w, words(keep))
    dense = ref.compress(wv, keep)[4]
    x, xv = tensor(rng.standard_normal((n, k)) * 2.0 ** 60, "bf16")
    xv = xv.copy()
    xv[:, :128] *= 2.0 ** -100            # blocks 2^100 apart in one row
    x = tensor(xv, "bf16")[0]
    clean = sms.spmm24_fp8(x, A, dtype=torch.float32)
    x[1, 5] = float("nan")
    y = sms.spmm24_fp8(x, A, dtype=torch.float32)
    sync()
    xd = ref.quant(xv)[2]
    close(clean, xd @ dense.T, np.abs(xd) @ np.abs(dense).T, sum_rel(k), torch.float32)
    assert bool((clean[:, 0] == 0).all())
    other = [i for i in range(n) if i != 1]
    assert torch.equal(y[other], clean[other])
    hit = torch.from_numpy((dense[:, 5] != 0)).cuda()
    assert bool(torch.isnan(y[1][hit]).all()) and int(hit.sum()) > 0


# Shapes that reach each tile size of the tiled kernels (256 x 256, 128 x 128, 128 x 64),
# ragged in every dimension.
TILED = [(4100, 4104, 260), (2900, 3012, 132), (1000, 4100, 388)]


def exact_product(x, w):
    """An integer-valued product on the GPU in fp64."""
    import torch
    return torch.from_numpy(x).cuda() @ torch.from_numpy(w).cuda().t()


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("n,m,k", TILED)
def test_spmm_tiles_exact(n, m, k, far):
    """far: some rows of X hold integers times 2^-80 in their first block and zeros (scale 1)
    behind it, so that scales more than 2^60 apart meet in one row."""
    import torch
    say("spmm tiles", n, m, k, far)
    rng = np.random.default_rng(n + m + k)
    keep = np.tile(ref.random24(rng, 64, k), (-(-m // 64), 1))[:m]
    w, wv = tensor(integers(rng, (m, k), 7) * powers_square(rng, m, k), "bf16")
    xv = integers(rng, (n, k), 7) * powers(rng, n, k)
    if far:
        rows = rng.choice(n, 40, replace=False)
        xv[rows, :128] *= 2.0 ** -80
        xv[rows, 128:] = 0
    x, xv = tensor(xv, "bf16")
    A, bad = sms.compress24_fp8(w, words(keep))
    buf = torch.full((n + 2, m + 4), 7.0, device="cuda")
    y = buf[1:n + 1, 4:m + 4]
    sms.spmm24_fp8(x, A, out=y)
    yb = sms.spmm24_fp8(x, A)
    sync()
    assert int(bad.item()) == 0
    assert torch.equal(y.double(), exact_product(xv, np.where(keep, wv, 0)))
    assert torch.equal(yb, y.bfloat16())
    y.fill_(7.0)
    assert bool((buf == 7.0).all())


def test_spmm_no_tokens():
    import torch
    rng = np.random.default_rng(2)
    w, _, keep = _weight(rng, 64, 64)
    A, _ = sms.compress24_fp8(w, words(keep))
    for x in (torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"),
              torch.empty((0, 64), dtype=torch.float32, device="cuda")):
        assert sms.spmm24_fp8(x, A).shape == (0, 64)
        assert sms.spmm24_fp8(sms.quant_fp8(x), A).shape == (0, 64)


@pytest.mark.parametrize("n", [1, 20, 300])
def test_spmm_operand_past_2_to_the_31(n):
    """An operand of 2.2e9 bytes: the rows at its end (and the block of 128 rows that
    ends past 2^31) against the reference."""
    import torch
    k, m = 4096, 1_074_000
    gen = torch.Generator(device="cuda").manual_seed(1)
    code = torch.randint(0, 0x7F, (m, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
    meta = torch.full((m, k // 32), 0x49D8E4C9, dtype=torch.int32, device="cuda")  # all six patterns
    scales = torch.randint(110, 120, (-(-m // 128), k // 128), dtype=torch.uint8, device="cuda", generator=gen)
    A = sms.Sparse24Fp8(code.view(torch.float8_e4m3fn), meta, scales.view(torch.float8_e8m0fnu), k)
    x, xv = tensor(np.random.default_rng(n).standard_normal((n, k)), "bf16")
    y = sms.spmm24_fp8(x, A, dtype=torch.float32)
    sync()
    xd = ref.quant(xv)[2]
    edge = 2 ** 31 // (k // 2) // 128 * 128
    for r0 in (0, edge, m - 96):
        r0 = r0 // 128 * 128
        r1 = min(m, r0 + 128)
        d = ref.expand(code[r0:r1].cpu().numpy(), meta[r0:r1].cpu().numpy().view(np.uint32),
                       scales[r0 // 128:r0 // 128 + 1].cpu().numpy())
        close(y[:, r0:r1], xd @ d.T, np.abs(xd) @ np.abs(d).T, sum_rel(k), torch.float32)


# ---- the dense product and the weight gradient --------------------------------

@pytest.mark.parametrize("p,q,k", [(1, 1, 1), (16, 16, 128), (60, 132, 300), (256, 260, 1001), (300, 520, 129),
                                   (512, 256, 512), (4, 700, 640)])
def test_gemm(p, q, k):
    import torch
    say("gemm", p, q, k)
    rng = np.random.default_rng(p + q + k)
    a, av = tensor(rng.standard_normal((p, k)) * np.exp(rng.standard_normal((p, 1))), "bf16")
    b, bv = tensor(rng.standard_normal((q, k)), "f32")
    ad, bd = ref.quant(av)[2], ref.quant(bv)[2]
    want, absum = ad @ bd.T, np.abs(ad) @ np.abs(bd).T
    keep = rng.random((p, q)) < 0.5
    keep[0] = False
    A, B = sms.quant_fp8(a), sms.quant_fp8(b)
    for dt in (torch.bfloat16, torch.float32):
        c = sms.gemm_fp8(A, B, dtype=dt)
        cm = sms.gemm_fp8(A, B, mask=words(keep), dtype=dt)
        buf = torch.full((p + 2, q + 5), 7.0, dtype=dt, device="cuda")
        part = buf[1:p + 1, 3:q + 3]
        sms.gemm_fp8(A, B, out=part)
        sync()
        close(c, want, absum, sum_rel(k), dt)
        assert torch.equal(cm, torch.where(torch.from_numpy(keep).cuda(), c, torch.zeros_like(c)))
        assert torch.equal(part, c)
        part.fill_(7.0)
        assert bool((buf == 7.0).all())


@pytest.mark.parametrize("p,q,k", [(1, 1, 1), (16, 16, 128), (60, 132, 300), (256, 260, 1001), (300, 520, 129),
                                   (512, 256, 512), (4, 700, 640), (257, 129, 900)])
def test_gemm_exact(p, q, k):
    import torch
    say("gemm exact", p, q, k)
    rng = np.random.default_rng(p * q + k)
    a, av = tensor(integers(rng, (p, k), 7) * powers(rng, p, k), "bf16")
    b, bv = tensor(integers(rng, (q, k), 7) * powers(rng, q, k), "bf16")
    c = sms.gemm_fp8(sms.quant_fp8(a), sms.quant_fp8(b), dtype=torch.float32)
    cb = sms.gemm_fp8(sms.quant_fp8(a), sms.quant_fp8(b))
    sync()
    assert np.array_equal(f64(c), av @ bv.T)
    assert torch.equal(cb, c.bfloat16())


@pytest.mark.parametrize("p,q,k", [(4100, 4104, 261), (2900, 3011, 130), (1000, 4099, 389)])
def test_gemm_tiles_exact(p, q, k):
    import torch
    say("gemm tiles", p, q, k)
    rng = np.random.default_rng(p + q + k)
    a, av = tensor(integers(rng, (p, k), 7) * powers(rng, p, k, 2), "bf16")
    b, bv = tensor(integers(rng, (q, k), 7) * powers(rng, q, k, 2), "bf16")
    keep = np.tile(rng.random((64, q)) < 0.5, (-(-p // 64), 1))[:p]
    A, B = sms.quant_fp8(a), sms.quant_fp8(b)
    buf = torch.full((p + 2, q + 4), 7.0, device="cuda")
    c = buf[1:p + 1, 4:q + 4]
    sms.gemm_fp8(A, B, mask=words(keep), out=c)
    cb = sms.gemm_fp8(A, B)
    sync()
    want = exact_product(av, bv)
    assert torch.equal(cb, want.float().bfloat16())
    assert torch.equal(c.double(), want * torch.from_numpy(keep).cuda())
    c.fill_(7.0)
    assert bool((buf == 7.0).all())


@pytest.mark.parametrize("p,q", [(24, 40), (300, 520), (4100, 4104)])
def test_gemm_no_tokens_gives_zeros(p, q):
    import torch
    x = torch.empty((0, q), dtype=torch.bfloat16, device="cuda")
    g = torch.empty((0, p), dtype=torch.bfloat16, device="cuda")
    out = torch.full((p, q), 5.0, device="cuda")
    sms.gemm_fp8(sms.quant_fp8(g, transpose=True), sms.quant_fp8(x, transpose=True), out=out)
    sync()
    assert bool((out == 0).all())


# ---- together: a masked layer, forward and backward -----------------------------

@pytest.mark.parametrize("n", [5, 40, 300])
def test_layer_gradients_against_formula_and_differences(n):
    """With small integers every 8-bit number, product and sum is exact (|sum| < 2^22), so
    the loss sum(G * (X W^T)) is exact too, and its central differences equal the gradients
    that the products give."""
    import torch
    rng = np.random.default_rng(n)
    m, k = 36, 140
    keep = ref.random24(rng, m, k)
    wv = np.where(keep, integers(rng, (m, k), 6), 0)
    xv, gv = integers(rng, (n, k), 6), integers(rng, (n, m), 3)
    mw = words(keep)

    def forward(xv, wv):
        A, _ = sms.compress24_fp8(tensor(wv, "bf16")[0], mw)
        return f64(sms.spmm24_fp8(tensor(xv, "bf16")[0], A, dtype=torch.float32))

    x, g = tensor(xv, "bf16")[0], tensor(gv, "bf16")[0]
    A, T, bad, bad_t = sms.compress24_fp8_both(tensor(wv, "bf16")[0], mw)
    (xq, xt), (gq, gt) = sms.quant_fp8_both(x), sms.quant_fp8_both(g)
    y = sms.spmm24_fp8(xq, A, dtype=torch.float32)
    dx = sms.spmm24_fp8(gq, T, dtype=torch.float32)
    dw = sms.gemm_fp8(gt, xt, mask=mw, dtype=torch.float32)
    sync()
    assert np.array_equal(f64(y), xv @ wv.T)
    assert np.array_equal(f64(dx), gv @ wv)
    assert np.array_equal(f64(dw), np.where(keep, gv.T @ xv, 0))
    for _ in range(6):
        i, j = rng.integers(n), rng.integers(k)
        step = np.zeros_like(xv)
        step[i, j] = 1
        diff = ((gv * forward(xv + step, wv)).sum() - (gv * forward(xv - step, wv)).sum()) / 2
        assert diff == f64(dx)[i, j]
        i, j = (int(v) for v in rng.choice(np.argwhere(keep)))
        step = np.zeros_like(wv)
        step[i, j] = 1
        diff = ((gv * forward(xv, wv + step)).sum() - (gv * forward(xv, wv - step)).sum()) / 2
        assert diff == f64(dw)[i, j]


def _train_step(w, x, g, m):
    A, T, _, _ = sms.compress24_fp8_both(w, m)
    xq, xt = sms.quant_fp8_both(x)
    gq, gt = sms.quant_fp8_both(g)
    return sms.spmm24_fp8(xq, A), sms.spmm24_fp8(gq, T), sms.gemm_fp8(gt, xt, mask=m)


@pytest.mark.parametrize("n,m,k", [(300, 512, 384), (512, 1024, 512)])
def test_step_from_mask_search_to_gradients(n, m, k):
    """The whole run: the library's own 2:4 mask, both operands under it, forward, data
    gradient, weight gradient; alone, replayed from a graph between eager calls, and
    interleaved on two streams."""
    import torch
    rng = np.random.default_rng(n)
    w, wv = tensor(0.02 * rng.standard_normal((m, k)), "bf16")
    mask, _ = sms.mask(w, 2, 4, 20.0, 50, 4)
    keep = sms.unpack(mask, k).cpu().numpy()
    x, xv = tensor(rng.standard_normal((n, k)), "bf16")
    g, gv = tensor(1e-3 * rng.standard_normal((n, m)), "bf16")
    y, dx, dw = _train_step(w, x, g, mask)
    sync()
    dense = ref.compress(wv, keep)[4][:, :k]
    xd, gd = ref.quant(xv)[2][:, :k], ref.quant(gv)[2][:, :m]
    close(y, xd @ dense.T, np.abs(xd) @ np.abs(dense).T, sum_rel(k), torch.bfloat16)
    close(dx, gd @ dense, np.abs(gd) @ np.abs(dense), sum_rel(m), torch.bfloat16)
    xt, gt = ref.quant(xv.T)[2], ref.quant(gv.T)[2]
    close(dw, np.where(keep, gt @ xt.T, 0), np.abs(gt) @ np.abs(xt).T, sum_rel(n), torch.bfloat16)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _train_step(w, x, g, mask)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        captured = _train_step(w, x, g, mask)
    for scale in (1.0, -2.0, 0.5, 1.0):
        x.copy_(tensor(scale * xv, "bf16")[0])
        graph.replay()
        sync()
        eager = _train_step(w, x, g, mask)
        sync()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager)), scale

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    inputs = [(w, x, g), (w.neg(), x.flip(0), g * 2)]
    alone = [_train_step(*t, mask) for t in inputs]
    sync()
    got = []
    for rep in range(3):
        for s, t in zip(streams, inputs):
            with torch.cuda.stream(s):
                got.append(_train_step(*t, mask))
    sync()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, alone[i % 2]))
    # the stream argument takes memory and runs on that stream
    one = sms.spmm24_fp8(x, sms.compress24_fp8(w, mask, stream=streams[0])[0], stream=streams[0])
    sync()
    assert torch.equal(one, alone[0][0])


def test_results_repeat():
    import torch
    rng = np.random.default_rng(4)
    w, _, keep = _weight(rng, 1000, 900)
    mw = words(keep)
    for n in (1, 16, 37, 300):
        x, g = tensor(rng.standard_normal((n, 900)), "bf16")[0], tensor(rng.standard_normal((n, 1000)), "bf16")[0]
        first = _train_step(w, x, g, mw) + (sms.spmm24_fp8(x, sms.compress24_fp8(w, mw)[0]),)
        for _ in range(3):
            again = _train_step(w, x, g, mw) + (sms.spmm24_fp8(x, sms.compress24_fp8(w, mw)[0]),)
            sync()
            assert all(torch.equal(a, b) for a, b in zip(first, again))


# ---- mixture of experts ----------------------------------------------------------

def _experts(rng, e, rows, k):
    ops, dense = [], []
    for _ in range(e):
        w, wv, keep = _weight(rng, rows, k)
        a, _ = sms.compress24_fp8(w, words(keep))
        ops.append(a)
        dense.append(ref.compress(wv, keep)[4][:, :k])
    import torch
    st = lambda i: torch.stack([o[i].view(torch.uint8) if i != 1 else o[i] for o in ops])
    return sms.Sparse24Fp8(st(0).view(torch.float8_e4m3fn), st(1), st(2).view(torch.float8_e8m0fnu), k), \
        np.stack(dense)


def _route(xv, rv, topk):
    logits = xv @ rv.T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :topk]
    top = np.take_along_axis(logits, ids, 1)
    p = np.exp(top - top[:, :1])
    return ids, p / p.sum(1, keepdims=True)


def _moe_reference(xv, ids, wts, gate, up, down):
    """y in 64 bits and a bound on the kernel's error before the last rounding.

    Products of bf16 numbers are exact in fp32; a sum of t of them in any order is off by
    at most t * 2^-24 of its magnitudes (the matrix cores' adds are counted the same).  silu has slope
    at most 1.1; exp, the division and two products: 2^-20.  The hidden entry loses at
    most 2^-16; the weights and the sum over experts: 2^-20."""
    n, d = xv.shape
    f = gate.shape[1]
    y, bound = np.zeros((n, d)), np.zeros((n, d))
    for t in range(n):
        for e, w in zip(ids[t], wts[t]):
            x = xv[t]
            g, u = gate[e] @ x, up[e] @ x
            eg, eu = d * 2.0 ** -24 * (np.abs(gate[e]) @ np.abs(x)), d * 2.0 ** -24 * (np.abs(up[e]) @ np.abs(x))
            silu = g / (1 + np.exp(-g))
            h = silu * u
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu) * eu + (2.0 ** -20 + 2.0 ** -16) * np.abs(h)
            a = np.abs(down[e])
            y[t] += w * (down[e] @ h)
            bound[t] += w * (a @ (1.01 * eh) + (f * 2.0 ** -24 + 2.0 ** -20) * (a @ np.abs(h)))
    return y, bound


@pytest.mark.parametrize("n,d,f,e,topk", [(1, 128, 128, 4, 2), (1, 260, 140, 8, 3), (2, 64, 36, 3, 1),
                                          (7, 516, 260, 16, 8), (17, 384, 132, 5, 5), (33, 256, 256, 4, 1),
                                          (64, 132, 388, 8, 2), (64, 256, 128, 2, 2), (5, 128, 64, 200, 16),
                                          (3, 128, 32, 1, 1), (64, 64, 36, 512, 3), (24, 1028, 1400, 12, 6)])
def test_moe(n, d, f, e, topk):
    import torch
    say("moe", n, d, f, e, topk)
    rng = np.random.default_rng(n * d + f)
    gate, gd = _experts(rng, e, f, d)
    up, ud = _experts(rng, e, f, d)
    down, dd = _experts(rng, e, d, f)
    x, xv = tensor(rng.standard_normal((n, d)), "bf16")
    r, rv = tensor(0.1 * rng.standard_normal((e, d)), "bf16")
    y, ids, wts = sms.moe24_fp8(x, r, gate, up, down, topk, return_routing=True)
    sync()
    wi, ww = _route(xv, rv, topk)
    assert np.array_equal(ids.cpu().numpy(), wi)
    assert np.abs(wts.cpu().numpy() - ww).max() <= 2.0 ** -20
    want, bound = _moe_reference(xv, wi, ww, gd, ud, dd)
    close(y, want, bound, 1.0, torch.bfloat16)
    # strided x, router and y: the same numbers, nothing else written
    xw = torch.zeros((n, d + 3), dtype=torch.bfloat16, device="cuda")
    rw = torch.zeros((e, d + 5), dtype=torch.bfloat16, device="cuda")
    xw[:, 1:d + 1], rw[:, 3:d + 3] = x, r
    buf = torch.full((n + 2, d + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    part = buf[1:n + 1, 2:d + 2]
    sms.moe24_fp8(xw[:, 1:d + 1], rw[:, 3:d + 3], gate, up, down, topk, out=part)
    sync()
    assert torch.equal(part, y)
    part.fill_(7.0)
    assert bool((buf == 7.0).all())


def test_moe_ties_nan_streams_and_graph():
    import torch
    rng = np.random.default_rng(11)
    n, d, f, e, topk = 20, 256, 128, 12, 4
    gate, gd = _experts(rng, e, f, d)
    up, ud = _experts(rng, e, f, d)
    down, dd = _experts(rng, e, d, f)
    x, xv = tensor(rng.standard_normal((n, d)), "bf16")
    rv = np.repeat(0.1 * rng.standard_normal((e // 4, d)), 4, 0)   # experts in four equal copies
    r, rv = tensor(rv, "bf16")
    y, ids, wts = sms.moe24_fp8(x, r, gate, up, down, topk, return_routing=True)
    sync()
    wi, ww = _route(xv, rv, topk)
    best = wi[:, :1] // 4 * 4
    assert np.array_equal(ids.cpu().numpy(), best + np.arange(4))   # the lowest of equal logits first
    want, bound = _moe_reference(xv, ids.cpu().numpy(), ww, gd, ud, dd)
    close(y, want, bound, 1.0, torch.bfloat16)
    # a NaN token leaves the others alone
    x2 = x.clone()
    x2[3, 7] = float("nan")
    y2, ids2, _ = sms.moe24_fp8(x2, r, gate, up, down, topk, return_routing=True)
    sync()
    other = [i for i in range(n) if i != 3]
    assert torch.equal(y2[other], y[other]) and bool(torch.isnan(y2[3]).all())
    assert ids2[3].tolist() == [0, 1, 2, 3]
    # no tokens
    assert sms.moe24_fp8(x[:0], r, gate, up, down, topk).shape == (0, d)
    # a graph replayed between eager calls, and calls on two streams
    graph = torch.cuda.CUDAGraph()
    xin = x.clone()
    with torch.cuda.graph(graph):
        captured = sms.moe24_fp8(xin, r, gate, up, down, topk)
    for k in range(3):
        xin.copy_(x.roll(k, 0))
        graph.replay()
        eager = sms.moe24_fp8(xin, r, gate, up, down, topk)
        sync()
        assert torch.equal(captured, eager) and torch.equal(eager, y.roll(k, 0))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for k in range(4):
        with torch.cuda.stream(streams[k % 2]):
            got.append(sms.moe24_fp8(x, r, gate, up, down, topk))
    got.append(sms.moe24_fp8(x, r, gate, up, down, topk, stream=streams[1]))
    sync()
    assert all(torch.equal(v, y) for v in got)


def test_refusals_on_tensors():
    """Every mismatch is refused before a launch."""
    import torch
    rng = np.random.default_rng(1)
    w, _, keep = _weight(rng, 64, 128)
    A, _ = sms.compress24_fp8(w, words(keep))
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        sms.spmm24_fp8(x[:, :64], A)                 # columns differ
    with pytest.raises(TypeError):
        sms.spmm24_fp8(x.half(), A)
    with pytest.raises(TypeError):
        sms.spmm24_fp8(x, (A.values, A.meta, A.scales))
    with pytest.raises(ValueError):
        sms.spmm24_fp8(x, A, out=torch.empty((4, 60), device="cuda"))
    with pytest.raises(ValueError):
        sms.spmm24_fp8(x, A, out=torch.empty((64, 4), device="cuda").t())
    with pytest.raises(ValueError):
        sms.spmm24_fp8(x, A._replace(values=A.values[:60]))
    with pytest.raises(ValueError):
        sms.spmm24_fp8(x, A._replace(scales=A.scales.view(torch.uint8)))
    with pytest.raises(ValueError):
        sms.gemm_fp8(sms.quant_fp8(x), sms.quant_fp8(x[:, :64].contiguous()))
    with pytest.raises(ValueError):
        sms.gemm_fp8(sms.quant_fp8(x), sms.quant_fp8(x), mask=words(keep))
    with pytest.raises(ValueError):
        sms.compress24_fp8(w, words(keep)[:32])
    with pytest.raises(ValueError):
        sms.quant_fp8(x.t())
    with pytest.raises(sms.TsenorError):             # rows not a multiple of 4
        sms.compress24_fp8(w[:62], words(keep)[:62].contiguous())
    st = lambda a: sms.Sparse24Fp8(a.values[None], a.meta[None], a.scales[None], a.k)
    r = torch.zeros((1, 128), dtype=torch.bfloat16, device="cuda")
    down, _ = sms.compress24_fp8(w, words(keep), transpose=True)
    for topk in (0, 2, 17):
        with pytest.raises((sms.TsenorError, RuntimeError)):
            sms.moe24_fp8(x, r, st(A), st(A), st(down), topk)
    with pytest.raises(sms.TsenorError):
        sms.moe24_fp8(torch.zeros((65, 128), dtype=torch.bfloat16, device="cuda"), r, st(A), st(A), st(down), 1)
    with pytest.raises(ValueError):
        sms.moe24_fp8(x, r, st(A), st(down), st(down), 1)


@pytest.mark.parametrize("n", [3, 16, 20, 70])
def test_spmm_out_beside_or_over_its_input(n):
    import torch
    rng = np.random.default_rng(n)
    w, _, keep = _weight(rng, 64, 64)
    A, _ = sms.compress24_fp8(w, words(keep))
    buf = torch.from_numpy(rng.standard_normal((n, 128)).astype(np.float32)).to(torch.bfloat16).cuda()
    want = sms.spmm24_fp8(buf[:, :64].clone(), A)
    with pytest.raises(ValueError):
        sms.spmm24_fp8(buf[:, :64], A, out=buf[:, :64])
    with pytest.raises(ValueError):
        sms.spmm24_fp8(buf[:, :64], A, out=buf[:, 32:96])
    sms.spmm24_fp8(buf[:, :64], A, out=buf[:, 64:])
    assert torch.equal(buf[:, 64:], want)
