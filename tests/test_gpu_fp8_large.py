"""GPU: the 8-bit operators at the ends of their sizes: rows of 2^23 bytes and more (past what the tiled
kernels take), operands, results and activations past 2^31 entries, the expert layer's limits.
Results are compared with sums in 64 bits, or with calls on a part of the same data."""
import pytest

import sparse_mask_search_amd as sms
from test_gpu_fp8 import say, sync

pytestmark = pytest.mark.gpu


def signs(shape, seed):
    """bf16 entries -1, 0 and 1 (exact in 8 bits; sums of 2^23 of them are exact in fp32)."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, shape, dtype=torch.int8, device="cuda", generator=gen).to(torch.bfloat16)


def halves(rows, cols, seed):
    """A 2:4 mask: the first or the last two of each group of four columns, and its complement two rows on."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pick = torch.randint(0, 2, (rows // 4, 1, cols // 4, 1), device="cuda", generator=gen, dtype=torch.int8)
    turn = torch.arange(4, device="cuda", dtype=torch.int8).view(1, 4, 1, 1) // 2
    keep = ((pick + turn) % 2 == torch.arange(4, device="cuda", dtype=torch.int8) // 2)
    return keep.reshape(rows, cols)


def packed(keep):
    """The words of a mask whose columns are a multiple of 32."""
    import torch
    rows, cols = keep.shape
    out = torch.zeros((rows, cols // 32), dtype=torch.int32, device="cuda")
    bits = keep.view(rows, cols // 32, 32)
    for j in range(32):
        out |= bits[:, :, j].to(torch.int32) << j
    return out


def product64(x, w):
    """x w^T in 64 bits, in pieces along k."""
    import torch
    y = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device="cuda")
    for k in range(0, x.shape[1], 1 << 20):
        y += x[:, k:k + (1 << 20)].double() @ w[:, k:k + (1 << 20)].double().t().contiguous()
    return y


@pytest.mark.parametrize("n", [1, 5, 66])
def test_spmm_rows_past_2_to_the_23(n):
    import torch
    say("spmm long rows", n)
    m, k = 68, (1 << 23) + 160
    w, x = signs((m, k), 1), signs((n, k), 2)
    keep = halves(m, k, 3)
    A, bad = sms.compress24_fp8(w, packed(keep))
    want = product64(x, w * keep)
    for X in (x, sms.quant_fp8(x)):
        y = sms.spmm24_fp8(X, A, dtype=torch.float32)
        sync()
        assert torch.equal(y.double(), want)
    assert int(bad.item()) == 0


def test_gemm_rows_past_2_to_the_23():
    import torch
    p, q, k = 68, 72, (1 << 23) + 130
    a, b = signs((p, k), 1), signs((q, k), 2)
    c = sms.gemm_fp8(sms.quant_fp8(a), sms.quant_fp8(b), dtype=torch.float32)
    sync()
    assert torch.equal(c.double(), product64(a, b))


def test_gemm_operand_and_result_past_2_to_the_31():
    """A of 2.2e9 bytes, then a result of 2.2e9 entries under a mask: their last rows equal the same rows alone."""
    import torch
    p, q, k = 66_900, 264, 32_896
    a, b = signs((p, k), 1), signs((q, k), 2)
    B = sms.quant_fp8(b)
    c = sms.gemm_fp8(sms.quant_fp8(a), B, dtype=torch.float32)
    for part in (slice(0, 300), slice(65_280, 65_700), slice(p - 300, p)):
        sync()
        assert torch.equal(c[part].double(), product64(a[part], b))
    del a, c
    say("result")
    p, q, k = 46_500, 47_008, 300
    a, b, keep = signs((p, k), 3), signs((q, k), 4), halves(p, q, 5)
    c = sms.gemm_fp8(sms.quant_fp8(a), sms.quant_fp8(b), mask=packed(keep))
    for part in (slice(0, 300), slice(45_600, 45_800), slice(p - 300, p)):
        want = product64(a[part], b) * keep[part]
        sync()
        assert torch.equal(c[part].double(), want)


@pytest.mark.parametrize("rows,cols", [(3, (1 << 30) + 5000), (300, (1 << 23) + 5000), ((1 << 24) + 300, 130)])
def test_quant_past_2_to_the_31(rows, cols):
    """The last rows, or the last columns, equal those of a call on them alone."""
    import torch
    say("quant", rows, cols)
    x = signs((rows, cols), 1)
    x *= torch.arange(1, 8, device="cuda", dtype=torch.bfloat16).repeat(-(-cols // 7))[:cols]
    parts = [(sms.quant_fp8(x), False)]
    if rows > 3:
        parts += zip(sms.quant_fp8_both(x), (False, True))
    sync()
    u8 = torch.uint8
    for part, turn in parts:
        if turn == (rows > cols):     # the long direction lies along the operand's rows: its last blocks
            at = (part.k - 1) // 128 * 128 - 512
            ref = sms.quant_fp8(x[at:] if turn else x[:, at:], transpose=turn)
            assert torch.equal(part.values.view(u8)[:, at:], ref.values.view(u8))
            assert torch.equal(part.scales.view(u8)[at // 128:], ref.scales.view(u8))
        else:                         # or along its lines
            ref = sms.quant_fp8(x[:, -600:] if turn else x[-600:], transpose=turn)
            n = ref.values.shape[0]
            assert torch.equal(part.values.view(u8)[-n:], ref.values.view(u8))
            assert torch.equal(part.scales.view(u8)[:, -n:], ref.scales.view(u8))


def test_compress_past_2_to_the_31():
    """W of 2.3e9 entries: the last blocks of 128 rows and of 128 columns equal those alone."""
    import torch
    rows, cols = 46_848, 49_152
    w, keep = signs((rows, cols), 1), halves(rows, cols, 2)
    w *= torch.arange(1, 8, device="cuda", dtype=torch.bfloat16).repeat(-(-cols // 7))[:cols]
    mask = packed(keep)
    a, t, bad, bad_t = sms.compress24_fp8_both(w, mask)
    ra, rt, _, _ = sms.compress24_fp8_both(w[-256:], mask[-256:])
    ca, ct, _, _ = sms.compress24_fp8_both(w[:, -256:], mask[:, -8:].contiguous())
    sync()
    u8 = torch.uint8
    assert int(bad.item()) == 0
    assert torch.equal(a.values.view(u8)[-256:], ra.values.view(u8)) and torch.equal(a.meta[-256:], ra.meta)
    assert torch.equal(a.scales.view(u8)[-2:], ra.scales.view(u8))
    assert torch.equal(t.values.view(u8)[:, -128:], rt.values.view(u8)) and torch.equal(t.meta[:, -8:], rt.meta)
    assert torch.equal(t.values.view(u8)[-256:], ct.values.view(u8)) and torch.equal(t.meta[-256:], ct.meta)
    assert torch.equal(a.values.view(u8)[:, -128:], ca.values.view(u8)) and torch.equal(t.scales.view(u8)[-2:], ct.scales.view(u8))


def _stack(e, rows, k, seed, only=None):
    """Experts' operand with entries -s, 0 and s for a power of two s (rows outside `only` are zero), and its fp64."""
    import torch
    w = torch.stack([signs((rows, k), seed + i) for i in range(e)]) * 2.0 ** -(k.bit_length() // 2)
    if only is not None:
        w *= torch.zeros((rows, 1), device="cuda").index_fill_(0, only, 1.0)
    keep = halves(e * rows, k, seed)
    a, bad = sms.compress24_fp8(w.bfloat16(), packed(keep).view(e, rows, k // 32))
    assert int(bad.item()) == 0
    return a, w.double() * keep.view(e, rows, k)


@pytest.mark.parametrize("n,d,f,e,topk", [(64, 64, 64, 512, 16), (64, 64, 32, 16, 16), (3, 1 << 20, 32, 2, 2),
                                          (3, 32, 1 << 20, 2, 2)])
def test_moe_limits(n, d, f, e, topk):
    """In the long sums at most 200 terms are not zero.  Bound on y: sums of t products in any order are
    off by at most t 2^-24 of their magnitudes, silu has slope at most 1.1, and exp, a division, the
    hidden vector's two bf16 numbers, the weights and their sum add 2^-15; then bf16 rounds (2^-8)."""
    import torch
    say("moe limits", n, d, f, e, topk)
    gen = torch.Generator(device="cuda").manual_seed(d + f)
    some = lambda size: torch.cat([torch.randint(0, size, (199,), device="cuda", generator=gen),
                                   torch.tensor([size - 1], device="cuda")])
    x = torch.randn((n, d), device="cuda", generator=gen)
    if d > 200:
        x *= torch.zeros(d, device="cuda").index_fill_(0, some(d), 1.0)
    x = x.bfloat16()
    (gate, gd), (up, ud) = _stack(e, f, d, 10), _stack(e, f, d, 20000, some(f) if f > 200 else None)
    down, dd = _stack(e, d, f, 40000)
    r = (torch.randn((e, d), device="cuda", generator=gen) * d ** -0.5).bfloat16()
    td, tf = min(d, 200), min(f, 200)
    y, ids, wts = sms.moe24_fp8(x, r, gate, up, down, topk, return_routing=True)
    sync()
    top, want_ids = (x.double() @ r.double().t()).sort(dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), want_ids[:, :topk])
    p = torch.softmax(top[:, :topk], 1)
    assert float((wts.double() - p).abs().max()) <= 2.0 ** -20
    xd = x.double()
    want, bound = torch.zeros_like(xd), torch.zeros_like(xd)
    for i in range(e):
        t, j = (ids == i).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        g, u = xd[t] @ gd[i].t(), xd[t] @ ud[i].t()
        eg, eu = (td * 2.0 ** -24 * (xd[t].abs() @ w[i].abs().t()) for w in (gd, ud))
        silu = g / (1 + torch.exp(-g))
        h = silu * u
        eh = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + 2.0 ** -15 * h.abs()
        w = p[t, j][:, None]
        want[t] += w * (h @ dd[i].t())
        bound[t] += w * ((1.01 * eh + (tf * 2.0 ** -24 + 2.0 ** -15) * h.abs()) @ dd[i].abs().t())
    err = (y.double() - want).abs()
    assert bool((err <= bound + 2.0 ** -8 * (want.abs() + bound) + 1e-38).all()), float(err.max())
