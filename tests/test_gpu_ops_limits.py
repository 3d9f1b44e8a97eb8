"""GPU: the dense operators of masked models at the ends of what they allow: every tile and its ring,
strides and alignments, rows of no expert, odd `ends`, NaN and infinities beside what is used, buffers
that stay as they were, streams, captured graphs, offsets past 32 bits.  Numbers are small integers
where results are compared bit for bit (tests/test_gpu_ops.py says why that is exact)."""
import numpy as np
import pytest

import ops_ref as ref
import sparse_mask_search_amd as sms
from test_gpu_ops import _clip_check, _int8_operands, bf16, ends_of, exactly, f64, ints, say, torch_type, words

pytestmark = pytest.mark.gpu

NAN = float("nan")


def spread(rng, total, experts):
    """Rows of experts, some without any."""
    share = rng.random(experts) * (rng.random(experts) < 0.8) + 1e-9
    return rng.multinomial(total, share / share.sum()).tolist()


# sizes that reach every form: few rows, 64 x 64 in both rings, 256 x 128, 256 x 256 (also with more
# tiles than workgroups), unaligned rows in 64 x 64 and 256 x 128; k that is no whole number of steps
FORMS = [
    (5, 64, 1024, 264), (40, 4, 4096, 520), (60, 1, 512, 1032), (300, 8, 512, 200), (700, 4, 512, 136),
    (2500, 6, 4096, 72), (9000, 5, 2304, 40), (9000, 3, 4096, 264), (3000, 2, 4097, 77), (200, 3, 333, 35),
]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows,experts,m,k", FORMS)
def test_grouped_mm_forms(rows, experts, m, k, transpose):
    say("forms mm", rows, experts, m, k, transpose)
    rng = np.random.default_rng(rows + m)
    counts = spread(rng, rows - 3, experts)
    x, xv = bf16(ints(rng, (rows, k)))
    w, wv = bf16(ints(rng, (experts, k, m) if transpose else (experts, m, k)))
    want, _ = ref.grouped_mm(xv, wv, np.cumsum(counts), transpose)
    exactly(sms.grouped_mm(x, w, ends_of(counts), transpose=transpose), want)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("rows,experts,m,k", [(300, 3, 200, 264), (2000, 4, 2048, 2304), (1500, 70, 512, 768),
                                              (5000, 9, 1280, 2056), (700, 5, 511, 1001), (90, 130, 256, 512)])
def test_grouped_wgrad_forms(rows, experts, m, k, masked):
    """More tiles than workgroups (the order of experts, two sets of mask words), more than 64 experts."""
    say("forms wgrad", rows, experts, m, k, masked)
    rng = np.random.default_rng(rows + k)
    counts = spread(rng, rows - 5, experts)
    x, xv = bf16(ints(rng, (rows, k)))
    dy, dyv = bf16(ints(rng, (rows, m)))
    keep = rng.random((experts, m, k)) < 0.5 if masked else None
    want, _ = ref.grouped_wgrad(dyv, xv, np.cumsum(counts), keep)
    exactly(sms.grouped_wgrad(dy, x, ends_of(counts), mask=words(keep) if masked else None), want)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,experts,m,k", [(2600, 1, 1792, 2056), (6000, 2, 1280, 1808), (1700, 5, 520, 1544)])
def test_grouped_wgrad_middle_tiles(rows, experts, m, k, dtype, masked):
    """128 x 128 with one tile and with more for a workgroup; 64 x 64 with more than one for a CU."""
    say("middle tiles", rows, experts, m, k, dtype, masked)
    rng = np.random.default_rng(rows + k)
    counts = spread(rng, rows - 5, experts)
    x, xv = bf16(ints(rng, (rows, k)))
    dy, dyv = bf16(ints(rng, (rows, m)))
    keep = rng.random((experts, m, k)) < 0.5 if masked else None
    want, _ = ref.grouped_wgrad(dyv, xv, np.cumsum(counts), keep)
    exactly(sms.grouped_wgrad(dy, x, ends_of(counts), mask=words(keep) if masked else None, dtype=torch_type(dtype)), want)


@pytest.mark.parametrize("rows,experts,m,k", [(2500, 6, 4096, 500), (9000, 3, 2304, 700), (300, 8, 512, 200)])
def test_gemm_int8_forms(rows, experts, m, k):
    import torch
    say("forms int8", rows, experts, m, k)
    rng = np.random.default_rng(rows)
    counts = spread(rng, rows - 3, experts)
    xv, xs, x = _int8_operands(rng, (), rows, k)
    av, as_, a = _int8_operands(rng, (experts,), m, k)
    got = sms.gemm_int8(x, a, ends=ends_of(counts), dtype=torch.float32)
    want = np.zeros((rows, m), np.float32)
    for e, (i, j) in enumerate(ref.bounds(np.cumsum(counts), rows)):
        sums = xv[i:j].astype(np.float64) @ av[e].astype(np.float64).T  # exact: below 2^53
        want[i:j] = sums.astype(np.float32) * xs[i:j, None] * as_[e][None]
    exactly(got, want)


@pytest.mark.parametrize("experts", [1, 63, 64, 65, 1000, 1024])
def test_many_experts(experts):
    rng = np.random.default_rng(experts)
    counts = rng.integers(0, 3, experts).tolist()
    x, xv = bf16(ints(rng, (sum(counts) + 2, 40)))
    w, wv = bf16(ints(rng, (experts, 72, 40)))
    want, _ = ref.grouped_mm(xv, wv, np.cumsum(counts), False)
    exactly(sms.grouped_mm(x, w, ends_of(counts)), want)
    dy, dyv = bf16(ints(rng, (sum(counts) + 2, 16)))
    exactly(sms.grouped_wgrad(dy, x, ends_of(counts)), ref.grouped_wgrad(dyv, xv, np.cumsum(counts))[0])


@pytest.mark.parametrize("ends", [[-5, 3, 100], [0, 0, 0], [2, 2, 2], [-1, -1, -1], [40, 40, 40], [1 << 31 - 1] * 3])
def test_ends_outside_the_rows(ends):
    import torch
    rng = np.random.default_rng(1)
    ends = [min(e, 2 ** 31 - 1) for e in ends]
    e = torch.tensor(ends, dtype=torch.int32).cuda()
    x, xv = bf16(ints(rng, (10, 64)))
    w, wv = bf16(ints(rng, (3, 32, 64)))
    dy, dyv = bf16(ints(rng, (10, 32)))
    exactly(sms.grouped_mm(x, w, e), ref.grouped_mm(xv, wv, ends, False)[0])
    exactly(sms.grouped_mm(dy, w, e, transpose=True), ref.grouped_mm(dyv, wv, ends, True)[0])
    exactly(sms.grouped_wgrad(dy, x, e), ref.grouped_wgrad(dyv, xv, ends)[0])


@pytest.mark.parametrize("rows,m,k", [(50, 64, 64), (400, 256, 64), (3000, 2048, 64), (50, 65, 33)])
def test_descending_ends(rows, m, k):
    """An entry below an earlier one counts as that one; what lies around the result stays as it was."""
    import torch
    rng = np.random.default_rng(2)
    few, many = [rows // 3, 3, rows // 2, 0, rows // 2 + 1, -7, rows - 2, 1], rng.integers(-5, rows, 130).tolist()
    for ends in (few, many, [rows + 9, 0, 5]):
        experts, e = len(ends), torch.tensor(ends, dtype=torch.int32).cuda()
        x, xv = bf16(ints(rng, (rows, k)))
        w, wv = bf16(ints(rng, (experts, m, k)))
        dy, dyv = bf16(ints(rng, (rows, m)))
        buf = torch.full((rows + 2, m + 8), 7.0, device="cuda", dtype=torch.bfloat16)
        exactly(sms.grouped_mm(x, w, e, out=buf[1:-1, :m]), ref.grouped_mm(xv, wv, ends, False)[0])
        assert (buf[0] == 7).all() and (buf[-1] == 7).all() and (buf[:, m:] == 7).all()
        exactly(sms.grouped_wgrad(dy, x, e), ref.grouped_wgrad(dyv, xv, ends)[0])


def _views(rng, shape, offset, pad):
    """A bf16 view with `pad` NaN columns behind each row, `offset` entries into its buffer, and its values."""
    import torch
    *lead, r, c = shape
    v = ints(rng, shape)
    flat = torch.full((offset + int(np.prod(lead, dtype=int)) * r * (c + pad) + 8,), NAN, device="cuda", dtype=torch.bfloat16)
    t = flat[offset:offset + int(np.prod(lead, dtype=int)) * r * (c + pad)].view(*lead, r, c + pad)[..., :c]
    t.copy_(torch.from_numpy(v.astype(np.float32)).cuda())
    return t, v


@pytest.mark.parametrize("offset,pad", [(0, 8), (8, 16), (1, 0), (3, 5), (4, 4), (0, 1)])
@pytest.mark.parametrize("rows,m,k", [(30, 96, 136), (500, 264, 200), (4500, 2304, 104)])
def test_strides_and_alignment(rows, m, k, offset, pad):
    """NaN beside the rows never enters, outputs are written where they belong only."""
    import torch
    say("strides", rows, m, k, offset, pad)
    rng = np.random.default_rng(offset * 7 + pad + rows)
    counts = spread(rng, rows - 2, 3)
    e = ends_of(counts)
    x, xv = _views(rng, (rows, k), offset, pad)
    w, wv = _views(rng, (3, m, k), offset, pad)
    wt, wtv = _views(rng, (3, k, m), offset, pad)
    dy, dyv = _views(rng, (rows, m), offset, pad)
    for t in (torch.bfloat16, torch.float32):
        out = torch.full((offset + rows * (m + pad) + 8,), 7.0, device="cuda", dtype=t)
        o = out[offset:offset + rows * (m + pad)].view(rows, m + pad)
        for ww, vv, tr in ((w, wv, False), (wt, wtv, True)):
            got = sms.grouped_mm(x, ww, e, transpose=tr, out=o[:, :m])
            assert got.data_ptr() == o.data_ptr()
            exactly(got, ref.grouped_mm(xv, vv, np.cumsum(counts), tr)[0])
            assert (o[:, m:] == 7).all() and (out[:offset] == 7).all() and (out[-8:] == 7).all()
        out = torch.full((3, m + 1, k + pad), 7.0, device="cuda", dtype=t)
        got = sms.grouped_wgrad(dy, x, e, out=out[:, :m, :k])
        exactly(got, ref.grouped_wgrad(dyv, xv, np.cumsum(counts))[0])
        assert (out[:, m:] == 7).all() and (out[:, :, k:] == 7).all()


@pytest.mark.parametrize("rows,m,k", [(12, 64, 64), (400, 128, 96), (4500, 2048, 72)])
def test_nan_stays_in_its_row(rows, m, k):
    import torch
    rng = np.random.default_rng(rows)
    counts = [rows // 3, 0, rows // 2]
    last = sum(counts)
    e = ends_of(counts)
    x, xv = bf16(ints(rng, (rows, k)))
    w, wv = bf16(ints(rng, (3, m, k)))
    dy, dyv = bf16(ints(rng, (rows, m)))
    want, _ = ref.grouped_mm(xv, wv, np.cumsum(counts), False)
    grad, _ = ref.grouped_wgrad(dyv, xv, np.cumsum(counts))
    # rows of no expert hold NaN, and the weights of the expert without rows
    x[last:], dy[last:], w[1] = NAN, NAN, NAN
    exactly(sms.grouped_mm(x, w, e), want)
    exactly(sms.grouped_wgrad(dy, x, e), grad)
    # one entry: its row of the product, its column of the owner's gradient
    x[rows // 3, 5] = NAN
    got, bad = f64(sms.grouped_mm(x, w, e)), np.arange(rows) == rows // 3
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], np.float64(torch.from_numpy(want[~bad]).to(torch.bfloat16).double()))
    got = f64(sms.grouped_wgrad(dy, x, e))
    assert np.isnan(got[2][:, 5]).all() and np.isfinite(np.delete(got[2], 5, 1)).all() and np.isfinite(got[:2]).all()
    # a masked place stays 0 whatever is there
    keep = np.ones((3, m, k), bool)
    keep[2, :, 5] = False
    got = f64(sms.grouped_wgrad(dy, x, e, mask=words(keep)))
    assert (got[2][:, 5] == 0).all() and np.isfinite(got).all()


def test_gemm_int8_nan_scale_and_strided_tokens():
    import torch
    rng = np.random.default_rng(9)
    for rows in (5, 40):
        x, _ = _views(rng, (rows, 300), 3, 5)
        x[2, 7] = float("inf")
        _, _, a = _int8_operands(rng, (), 64, 300)
        got = sms.gemm_int8(x, a, dtype=torch.float32)
        q = sms.quant_int8(x.contiguous())
        exactly(got, ref.gemm_int8(q.values.cpu().numpy(), q.scales.cpu().numpy(), a.values.cpu().numpy(), a.scales.cpu().numpy()))
        assert torch.isnan(got[2]).all() and torch.isfinite(got[:2]).all() and torch.isfinite(got[3:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quant_int8_stacks_and_views(dtype):
    import torch
    rng = np.random.default_rng(4)
    big = torch.from_numpy(rng.standard_normal((5, 9, 333)).astype(np.float32)).cuda().to(torch_type(dtype))
    for v in (big, big[1:4], big[:, 2:7], big[:, :, 1:301], big[:, :, :1], big[2:3], big[0], big[0, :, 3:], big[0, 4:5], big[:, 3:4]):
        q = sms.quant_int8(v)
        values, scales = ref.quant_int8(v.to(torch.float32).cpu().numpy())
        assert np.array_equal(q.values.cpu().numpy(), values) and np.array_equal(q.scales.cpu().numpy(), scales)
    assert sms.quant_int8(big[:0]).values.shape == (0, 9, 384) and sms.quant_int8(big[0, :0]).scales.shape == (0,)


def test_stacks_of_single_rows():
    """A matrix of one row may have any row stride: here more than that from matrix to matrix."""
    import torch
    rng = np.random.default_rng(6)
    counts = [3, 0, 5]
    e = ends_of(counts)
    x, xv = bf16(ints(rng, (8, 40)))
    y, yv = bf16(ints(rng, (8, 1)))
    w, wv = bf16(ints(rng, (7, 3, 40)))
    w, wv = w.transpose(0, 1)[:, 2:3], wv.transpose(1, 0, 2)[:, 2:3]
    assert w.stride(1) > w.stride(0)
    exactly(sms.grouped_mm(x, w, e), ref.grouped_mm(xv, wv, np.cumsum(counts), False)[0])
    exactly(sms.grouped_mm(y, w, e, transpose=True), ref.grouped_mm(yv, wv, np.cumsum(counts), True)[0])
    out = torch.full((7, 3, 40), 5.0, device="cuda", dtype=torch.float32)
    exactly(sms.grouped_wgrad(y, x, e, out=out.transpose(0, 1)[:, 2:3]), ref.grouped_wgrad(yv, xv, np.cumsum(counts))[0])
    assert (out[:2] == 5).all() and (out[3:] == 5).all()
    q, (values, scales) = sms.quant_int8(w), ref.quant_int8(wv.astype(np.float32))
    assert np.array_equal(q.values.cpu().numpy(), values) and np.array_equal(q.scales.cpu().numpy(), scales)


def test_longest_integer_rows():
    """k = 2^17 of 127 * 127: 2^17 * 127^2 = 2114060288 < 2^31."""
    import torch
    k = 1 << 17
    v = torch.full((2, k), 127, dtype=torch.int8, device="cuda")
    v[1] = -127
    one = torch.ones(2, device="cuda")
    a = sms.DenseInt8(v, one, k)
    exactly(sms.gemm_int8(a, a, dtype=torch.float32), np.float32(127 * 127) * np.float32(k) * np.array([[1, -1], [-1, 1]]))
    x = torch.ones(1, k, device="cuda", dtype=torch.bfloat16)
    x[0, 5] = -2
    q = sms.quant_int8(x)
    assert int(q.values[0, 5]) == -127 and int(q.values[0, 4]) == 64  # 63.5, a tie
    with pytest.raises(sms.TsenorError):
        sms.quant_int8(torch.ones(1, k + 1, device="cuda"))


def test_offsets_past_32_bits():
    """Tensors of more than 2^32 bytes and 2^31 entries: the last expert's weights, the last rows."""
    import torch
    experts, m, k = 65, 8192, 4104
    w = torch.zeros(experts, m, k, device="cuda", dtype=torch.bfloat16)
    rng = np.random.default_rng(3)
    tail, tv = bf16(ints(rng, (m, k)))
    w[-1] = tail
    x, xv = bf16(ints(rng, (9, k)))
    counts = [0] * (experts - 2) + [2, 7]
    got = sms.grouped_mm(x, w, ends_of(counts))
    want = np.zeros((9, m))
    want[2:] = xv[2:] @ tv.T
    exactly(got, want)
    mask = torch.zeros(experts, m, (k + 31) // 32, device="cuda", dtype=torch.int32)
    mask[-1] = -1
    dy, dyv = bf16(ints(rng, (9, m)))
    dw = sms.grouped_wgrad(dy, x, ends_of(counts), mask=mask, out=w)
    assert float(dw[:-1].abs().max()) == 0.0
    exactly(dw[-1], dyv[2:].T @ xv[2:])
    norm = sms.grad_norm([dw], masks=[mask])
    total = float((dw[-1].double() ** 2).sum())
    assert abs(float(norm) - total ** 0.5) <= total ** 0.5 * 2.0 ** -23


def test_clip_keeps_non_finite_rules():
    import torch
    g = [torch.ones(3, 40, device="cuda"), torch.ones(1000, device="cuda", dtype=torch.bfloat16)]
    keep = np.ones((3, 40), bool)
    keep[1, 7] = False
    mask = [words(keep), None]
    g[0][1, 7] = NAN  # removed: neither in the norm nor in the result
    norm = sms.clip_grads(g, 1.0, masks=mask)
    assert abs(float(norm) - 1119 ** 0.5) < 1e-5 and torch.isfinite(g[0]).all() and float(g[0][1, 7]) == 0.0
    g[1][3] = float("inf")
    assert float(sms.clip_grads(g, 1.0, masks=mask)) == float("inf")
    assert bool(torch.isnan(g[1][3])) and float(g[0].abs().max()) == 0.0 and float(g[0][1, 7]) == 0.0
    g[1][3] = NAN
    norm = sms.clip_grads(g, 1.0, masks=mask)
    assert np.isnan(float(norm)) and torch.isnan(g[1]).all() and float(g[0][1, 7]) == 0.0
    # the largest and smallest numbers: squares in 64 bits
    big = torch.full((70000,), 3e38, device="cuda")
    assert float(sms.clip_grads([big[:1]], 1.5e38)) == float(np.float32(3e38)) and float(big[0]) <= 1.5e38 * (1 + 2.0 ** -22)
    assert float(sms.grad_norm([big])) == float("inf")  # 7.9e40 has no fp32
    tiny = torch.full((10000,), 1e-30, device="cuda")
    assert abs(float(sms.grad_norm([tiny])) - 1e-28) <= 1e-28 * 2.0 ** -22


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_clip_layouts(dtype):
    """Views, columns, odd offsets, masks over rows of any length, empty tensors; what lies around stays."""
    import torch
    rng = np.random.default_rng(8)
    t = torch_type(dtype)
    base = torch.from_numpy(rng.standard_normal((60, 800)).astype(np.float32)).cuda().to(t)
    for masked in (False, True):
        buf = base.clone()
        views = [buf[:7, :33], buf[7:20, 1:90], buf[20:25, :800], buf[25:26, 3:600], buf[30:40, 8:408], buf[41:42, 5:6],
                 buf[:0], buf[45:50, 100:]]
        if not masked:
            views += [buf[50:58, 16:80].t(), buf[58, 1:], buf[59, 0]]
        keeps = [rng.random(tuple(v.shape)) < 0.5 if masked and v.dim() == 2 else None for v in views]
        masks = [None if k is None else words(k) for k in keeps]
        before = [v.clone() for v in views]
        norm = sms.grad_norm(views, masks=masks)
        got = sms.clip_grads(views, 1.0, masks=masks)
        assert float(got) == float(norm)
        _clip_check(before, views, keeps, 1.0, norm)
        inside = torch.zeros_like(base, dtype=torch.bool)
        rest = buf.clone()
        for v in views:
            v.fill_(NAN)
        inside = torch.isnan(buf)
        assert torch.equal(rest[~inside], base[~inside])
    # an out of other strides
    src, dst = base[:10, :48], torch.zeros(10, 60, device="cuda", dtype=t)[:, 4:52]
    norm = sms.clip_grads([src.contiguous()], 2.0, out=[dst])
    _clip_check([src], [dst], [None], 2.0, norm)


def test_clip_in_place_below_the_limit_writes_nothing_else():
    import torch
    g = torch.randn(40, 100, device="cuda")
    h = g.clone()
    sms.clip_grads([g], float("inf"))
    assert torch.equal(g, h)
    keep = np.random.default_rng(0).random((40, 100)) < 0.5
    sms.clip_grads([g], float("inf"), masks=[words(keep)])
    assert torch.equal(g.cpu(), torch.where(torch.from_numpy(keep), h.cpu(), torch.zeros(())))


def test_many_tensors_and_repeatability():
    """More tensors than a launch takes; the same bits on every run."""
    import torch
    g = [torch.randn(37 + i, 16 + i % 9, device="cuda") for i in range(301)]
    norms = {float(sms.grad_norm(g)) for _ in range(5)}
    assert len(norms) == 1
    want = float(torch.stack([x.double().square().sum() for x in g]).sum().sqrt())
    assert abs(norms.pop() - want) <= want * (2.0 ** -24 + 1e-9)
    out = [torch.empty_like(x) for x in g]
    norm = sms.clip_grads(g, 3.0, out=out)
    _clip_check(g, out, [None] * len(g), 3.0, norm)


def _operands(rng, rows=700, experts=4, m=512, k=264):
    counts = spread(rng, rows, experts)
    x, _ = bf16(ints(rng, (rows, k)))
    w, _ = bf16(ints(rng, (experts, m, k)))
    dy, _ = bf16(ints(rng, (rows, m)))
    return x, w, dy, ends_of(counts)


def _everything(x, w, dy, ends, out=None):
    """A layer's forward, backward, clipping and integer form."""
    import torch
    out = out or {}
    y = sms.grouped_mm(x, w, ends, out=out.get("y"))
    dx = sms.grouped_mm(dy, w, ends, transpose=True, out=out.get("dx"))
    dw = sms.grouped_wgrad(dy, x, ends, out=out.get("dw"))
    clipped = out.get("clipped") or [torch.empty_like(dw), torch.empty_like(dx)]
    norm = sms.clip_grads([dw, dx], 1.0, out=clipped)
    y8 = sms.gemm_int8(x, sms.quant_int8(w), ends=ends, out=out.get("y8"))
    one = sms.gemm_int8(x[:3], sms.quant_int8(w[0]), out=out.get("one"))
    return {"y": y, "dx": dx, "dw": dw, "clipped": clipped, "norm": norm, "y8": y8, "one": one}


def _same(a, b):
    import torch
    for key in a:
        for u, v in zip(a[key] if isinstance(a[key], list) else [a[key]], b[key] if isinstance(b[key], list) else [b[key]]):
            assert torch.equal(u, v), key


def test_two_streams_at_once():
    import torch
    sets = [_operands(np.random.default_rng(s)) for s in (1, 2)]
    want = [_everything(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _everything(*sets[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        _same(a, b)
    y = sms.grouped_mm(sets[0][0], sets[0][1], sets[0][3], stream=streams[1])
    norm = sms.grad_norm([sets[0][0]], stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]["y"]) and float(norm) == float(sms.grad_norm([sets[0][0]]))


def test_captured_and_replayed():
    """One capture of the whole layer, replayed on changed inputs and `ends`, eager work between."""
    import torch
    x, w, dy, ends = _operands(np.random.default_rng(5))
    _everything(x, w, dy, ends)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = _everything(x, w, dy, ends)
    for seed in (6, 7, 8, 9):
        a, b, c, d = _operands(np.random.default_rng(seed))
        for to, fresh in ((x, a), (w, b), (dy, c), (ends, d)):
            to.copy_(fresh)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _same(held, _everything(x, w, dy, ends))
        torch.cuda.synchronize()


def test_two_graphs_with_their_own_results():
    import torch
    sets = [_operands(np.random.default_rng(s), rows=90, m=128, k=64) for s in (1, 2)]
    want = [_everything(*s) for s in sets]
    graphs, held = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(_everything(*s))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, held):
            _same(a, b)
        sms.grad_norm([sets[0][0]])
        torch.cuda.synchronize()


def test_repeatable_bits():
    import torch
    rng = np.random.default_rng(12)
    x = torch.from_numpy(rng.standard_normal((3000, 1000)).astype(np.float32)).cuda().to(torch.bfloat16)
    w = torch.from_numpy(rng.standard_normal((5, 2048, 1000)).astype(np.float32)).cuda().to(torch.bfloat16)
    dy = torch.from_numpy(rng.standard_normal((3000, 2048)).astype(np.float32)).cuda().to(torch.bfloat16)
    e = ends_of(spread(rng, 3000, 5))
    first = _everything(x, w, dy, e)
    for _ in range(3):
        _same(first, _everything(x, w, dy, e))


def test_refused_on_the_device():
    """What the binding finds out before a launch."""
    import torch
    x, w, dy, ends = _operands(np.random.default_rng(1), rows=40, m=64, k=32)
    y = sms.grouped_mm(x, w, ends)
    bad_value = [
        lambda: sms.grouped_mm(x, w[:, :, :-1], ends), lambda: sms.grouped_mm(x, w, ends[:-1]), lambda: sms.grouped_mm(x, w, ends.long()),
        lambda: sms.grouped_mm(x, w, ends.cpu()), lambda: sms.grouped_mm(x, w, ends, out=y[:-1]), lambda: sms.grouped_mm(x, w[0], ends),
        lambda: sms.grouped_mm(x, w, ends, out=y.t()), lambda: sms.grouped_mm(x.t(), w, ends),
        lambda: sms.grouped_mm(x, w, ends, out=x.view(-1)[:1].expand(40, 64)),
        lambda: sms.grouped_mm(x, w, ends, out=y[1:]), lambda: sms.grouped_wgrad(dy[:-1], x, ends),
        lambda: sms.grouped_wgrad(dy, x, ends, mask=torch.zeros(4, 64, 2, dtype=torch.int32, device="cuda")),
        lambda: sms.grouped_wgrad(dy, x, ends, out=torch.empty(4, 64, 33, device="cuda")[:3]),
        lambda: sms.grouped_wgrad(dy, x, ends, out=torch.empty(4, 64, 32, device="cuda"), dtype=torch.bfloat16),
        lambda: sms.gemm_int8(x, sms.quant_int8(w)), lambda: sms.gemm_int8(x, sms.quant_int8(w[0]), ends=ends),
        lambda: sms.gemm_int8(x[:, :-1], sms.quant_int8(w[0])), lambda: sms.quant_int8(x[0]), lambda: sms.quant_int8(x[:, :0]),
        lambda: sms.clip_grads([x, x], 1.0), lambda: sms.clip_grads([x, x[3:5]], 1.0), lambda: sms.clip_grads([x], 1.0, masks=[]),
        lambda: sms.clip_grads([x], 1.0, out=[]),
    ]
    out = sms.grouped_mm(dy, w, ends, transpose=True, out=torch.empty_like(x))  # a plain one passes
    assert out.shape == x.shape
    for i, call in enumerate(bad_value):
        with pytest.raises((ValueError, RuntimeError)):
            print("[refused]", i, flush=True)
            call()
    for call in (lambda: sms.grouped_mm(x.float(), w, ends), lambda: sms.grouped_mm(x, w.float(), ends),
                 lambda: sms.grouped_mm(x, w, ends, dtype=torch.float16), lambda: sms.gemm_int8(x, w[0]), lambda: sms.quant_int8(x.half()),
                 lambda: sms.clip_grads([x.double()], 1.0), lambda: sms.clip_grads([x, None], 1.0), lambda: sms.clip_grads([], 1.0),
                 lambda: sms.grad_norm(x for x in [x])):
        with pytest.raises((TypeError, ValueError)):
            call()
    for call in (lambda: sms.clip_grads([x], -1.0), lambda: sms.clip_grads([x], NAN),
                 lambda: sms.grouped_mm(x, w[:1].expand(1025, -1, -1), ends[:1].expand(1025).contiguous())):
        with pytest.raises(sms.TsenorError):
            call()


def test_outputs_beside_inputs_of_one_buffer():
    import torch
    rng = np.random.default_rng(3)
    buf = torch.zeros(50, 200, device="cuda", dtype=torch.bfloat16)
    xv = ints(rng, (50, 64))
    buf[:, :64] = torch.from_numpy(xv.astype(np.float32)).cuda()
    w, wv = bf16(ints(rng, (2, 128, 64)))
    got = sms.grouped_mm(buf[:, :64], w, ends_of([20, 30]), out=buf[:, 64:192])
    exactly(got, ref.grouped_mm(xv, wv, [20, 50], False)[0])
    with pytest.raises(ValueError, match="overlaps"):
        sms.grouped_mm(buf[:, :64], w, ends_of([20, 30]), out=buf[:, 63:191])
    with pytest.raises(ValueError, match="overlaps"):
        sms.grouped_wgrad(buf[:, :8], buf[:, 8:24], ends_of([20, 30]), out=buf.view(-1)[:256].view(2, 8, 16))


def test_no_rows():
    import torch
    w = torch.ones(3, 64, 32, device="cuda", dtype=torch.bfloat16)
    ends = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, dy = w.new_empty(0, 32), w.new_empty(0, 64)
    assert sms.grouped_mm(x, w, ends).shape == (0, 64) and sms.grouped_mm(dy, w, ends, transpose=True).shape == (0, 32)
    assert float(sms.grouped_wgrad(dy, x, ends).abs().max()) == 0.0
    assert sms.gemm_int8(x, sms.quant_int8(w), ends=ends).shape == (0, 64)
    assert float(sms.grad_norm([w.new_empty(0, 5)])) == 0.0
