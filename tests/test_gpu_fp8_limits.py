"""GPU: the 8-bit operators where their numbers' range ends."""
import numpy as np
import pytest

import fp8_ref as ref
import sparse_mask_search_amd as sms
from test_gpu_fp8 import _experts, _moe_reference, bytes_of, close, f64, integers, say, sync, tensor, words

pytestmark = pytest.mark.gpu


# ---- the expert layer's router -------------------------------------------------

@pytest.mark.parametrize("n", [1, 6])
def test_moe_router_products_outside_fp32(n):
    """Logits of 2^140, -2^140, 2^-160 and 0: all numbers in 64 bits, none of the first three in 32."""
    import torch
    say("router", n)
    rng = np.random.default_rng(n)
    d, f = 64, 64
    gate, up, down = _experts(rng, 4, f, d)[0], _experts(rng, 4, f, d)[0], _experts(rng, 4, d, f)[0]
    x, r = torch.zeros((n, d)), torch.zeros((4, d))
    x[:, 0], x[:, 1] = 2.0 ** 70, 2.0 ** -80
    r[1, 0], r[2, 0], r[3, 1] = 2.0 ** 70, -2.0 ** 70, 2.0 ** -80
    _, ids, wts = sms.moe24_fp8(x.bfloat16().cuda(), r.bfloat16().cuda(), gate, up, down, 4, return_routing=True)
    sync()
    assert ids.tolist() == [[1, 3, 0, 2]] * n
    assert wts.tolist() == [[1.0, 0.0, 0.0, 0.0]] * n


def test_moe_topk_past_32_bits_is_refused():
    """The library takes an int: 2^32 + 1 must not arrive there as 1."""
    import torch
    rng = np.random.default_rng(1)
    gate, up, down = _experts(rng, 2, 64, 64)[0], _experts(rng, 2, 64, 64)[0], _experts(rng, 2, 64, 64)[0]
    x, r = torch.zeros((1, 64), dtype=torch.bfloat16).cuda(), torch.zeros((2, 64), dtype=torch.bfloat16).cuda()
    for topk in (2 ** 32 + 1, -2 ** 32 + 1, 2 ** 31, -1, 0, 3):
        for routing in (False, True):
            with pytest.raises(sms.TsenorError):
                sms.moe24_fp8(x, r, gate, up, down, topk, return_routing=routing)
    assert sms.moe24_fp8(x, r, gate, up, down, 1).shape == (1, 64)


# ---- results over operands -----------------------------------------------------------

def test_out_over_any_operand_is_refused():
    """The products read their operands while others of their workgroups write already."""
    import torch
    rng = np.random.default_rng(2)
    n = m = 64
    w, _ = tensor(rng.standard_normal((m, 256)), "bf16")
    A, _ = sms.compress24_fp8(w, words(ref.random24(rng, m, 256)))
    x, _ = tensor(rng.standard_normal((n, 256)), "bf16")
    X, B = sms.quant_fp8(x), sms.quant_fp8(w)
    mask = torch.full((n, 2), -1, dtype=torch.int32, device="cuda")
    over = lambda t, cols=64: t.view(torch.bfloat16)[:, :cols]
    for out in (over(X.values), over(A.values)):
        with pytest.raises(ValueError, match="overlaps"):
            sms.spmm24_fp8(X, A, out=out)
    with pytest.raises(ValueError, match="overlaps"):
        sms.spmm24_fp8(x, A, out=over(A.values))
    for out in (over(X.values), over(B.values)):
        with pytest.raises(ValueError, match="overlaps"):
            sms.gemm_fp8(X, B, out=out)
    words4 = torch.full((n, 64), -1, dtype=torch.int32, device="cuda").view(-1)[:n * 2].view(n, 2)
    with pytest.raises(ValueError, match="overlaps"):
        sms.gemm_fp8(X, B, mask=words4, out=torch.as_strided(words4, (n, 64), (64, 1)).view(torch.float32))
    gate, up, down = (_experts(rng, n, 64, 64)[0] for _ in range(3))
    r, _ = tensor(rng.standard_normal((n, 64)), "bf16")
    t = x[:, :64].contiguous()
    for out in (r, t, gate.values.view(torch.bfloat16).view(n, -1)[:, :64], down.meta.view(torch.bfloat16).view(n, -1)[:, :64]):
        with pytest.raises(ValueError, match="overlaps"):
            sms.moe24_fp8(t, r, gate, up, down, 2, out=out)
    # beside them it is taken, and nothing of the operand changes
    buf = torch.zeros((n, 128), dtype=torch.bfloat16, device="cuda")
    buf[:, 64:] = r
    want = sms.moe24_fp8(t, r, gate, up, down, 2)
    got = sms.moe24_fp8(t, buf[:, 64:], gate, up, down, 2, out=buf[:, :64])
    sync()
    assert torch.equal(got, want) and torch.equal(buf[:, 64:], r)
    assert torch.equal(sms.gemm_fp8(X, B, mask=mask, out=torch.empty((n, m), device="cuda")),
                       sms.gemm_fp8(X, B, dtype=torch.float32))


# ---- unused slots of a group -------------------------------------------------------

@pytest.mark.parametrize("n", [3, 40, 300])
def test_spmm_nan_at_removed_positions(n):
    """A group with fewer than two kept entries has unused slots: zeros that point at the positions
    0 and 1 of an empty group, at 3 beside one kept entry (2 if that is itself at 3).  A NaN
    there reaches the result, at the other removed positions it does not."""
    import torch
    say("removed positions", n)
    rng = np.random.default_rng(n)
    m, k = 132, 260
    keep = ref.random24(rng, m, k)
    keep[:5] = False                       # row 4 stays empty
    for p in range(4):
        keep[p, p::4] = True               # row p keeps position p of each group
    w, _ = tensor(integers(rng, (m, k), 7) + 8, "bf16")
    A, _ = sms.compress24_fp8(w, words(keep))
    wv = f64(w) * keep
    xv = integers(rng, (n, k), 7)
    reach = np.array([[1, 0, 0, 1], [0, 1, 0, 1], [0, 0, 1, 1], [0, 0, 1, 1], [1, 1, 0, 0]], bool)
    full = np.concatenate([np.tile(reach, (1, k // 4)), keep[5:]])
    for j in (0, 1, 2, 3, 130, 131, 256, 259):
        x = torch.from_numpy(xv.astype(np.float32)).bfloat16().cuda()
        x[1, j] = float("nan")
        for X in (x, sms.quant_fp8(x)):
            y = sms.spmm24_fp8(X, A, dtype=torch.float32)
            sync()
            got = f64(y)
            assert np.array_equal(np.isnan(got[1]), full[:, j]), j
            clean = np.ones_like(got, bool)
            clean[1] = ~full[:, j]
            assert np.array_equal(got[clean], (xv @ wv.T)[clean])   # small integers: exact


@pytest.mark.parametrize("j", [40, 41, 42, 43])
def test_moe_infinite_hidden_entry_at_removed_positions(j):
    """Entry j of the hidden vector is infinite, the others are 0.  Row 0 of down is empty: it
    meets the infinity (0 * inf) where its unused slots point at it, else it is 0."""
    import torch
    rng = np.random.default_rng(j)
    d = f = 128
    gate, _ = sms.compress24_fp8(torch.ones((1, f, d)).cuda(), words(ref.random24(rng, f, d))[None])
    u = torch.zeros((1, f, d))
    u[0, j] = 2.0 ** 120
    up, _ = sms.compress24_fp8(u.cuda(), words(ref.random24(rng, f, d))[None])
    keep = ref.random24(rng, d, f)
    keep[0] = False
    down, _ = sms.compress24_fp8(torch.ones((1, d, f)).cuda(), words(keep)[None])
    x = torch.full((1, d), 16.0, dtype=torch.bfloat16, device="cuda")
    y = sms.moe24_fp8(x, torch.zeros((1, d), dtype=torch.bfloat16, device="cuda"), gate, up, down, 1)
    sync()
    got = f64(y)[0]
    assert np.array_equal(np.isinf(got), keep[:, j])
    assert np.isnan(got[0]) == (j % 4 < 2)
    rest = ~keep[:, j]
    rest[0] = j % 4 >= 2
    assert (got[rest] == 0).all()


# ---- the expert layer at the ends of the scales --------------------------------------

@pytest.mark.parametrize("byte", [0, 1, 2, 9, 12, 60, 200, 245])
@pytest.mark.parametrize("which", ["gate", "up", "down"])
@pytest.mark.filterwarnings("ignore:overflow encountered in exp")   # silu of a large negative number
def test_moe_scales_at_the_ends(which, byte):
    """One operand's blocks all have the scale 2^(byte - 127).  Weights become bf16 numbers,
    subnormal ones too, so the lowest scales lose what lies below 2^-133 of a weight (at most
    2^-134 by rounding) and nothing else; the tokens and the other operands bring the layer back
    into range."""
    import torch
    say("moe scales", which, byte)
    rng = np.random.default_rng(byte)
    n, d, f = 3, 256, 132
    ops = {"gate": _experts(rng, 1, f, d)[0], "up": _experts(rng, 1, f, d)[0], "down": _experts(rng, 1, d, f)[0]}
    shift = max(-100, min(100, 117 - byte)) if which != "down" else 0
    for name, a in ops.items():
        s = a.scales.view(torch.uint8)
        s.fill_(byte if name == which else 117 if name == "down" else max(1, 117 - shift))
    x, xv = tensor(rng.standard_normal((n, d)) * 2.0 ** shift, "bf16")
    r = torch.zeros((1, d), dtype=torch.bfloat16, device="cuda")
    y = sms.moe24_fp8(x, r, ops["gate"], ops["up"], ops["down"], 1)
    sync()
    dense = {name: ref.expand(bytes_of(a.values)[0], a.meta[0].cpu().numpy().view(np.uint32),
                              bytes_of(a.scales)[0])[None] for name, a in ops.items()}
    gate, up, down = dense["gate"][:, :, :d], dense["up"][:, :, :d], dense["down"][:, :, :f]
    want, bound = _moe_reference(xv, np.zeros((n, 1), int), np.ones((n, 1)), gate, up, down)
    g, u = xv @ gate[0].T, xv @ up[0].T
    silu, lost = g / (1 + np.exp(-g)), 2.0 ** -134
    reach = lost * np.abs(xv).sum(1, keepdims=True)
    if which == "down":
        bound = bound + lost * np.abs(silu * u).sum(1, keepdims=True)
    else:
        dh = 1.1 * reach * np.abs(u) if which == "gate" else reach * np.abs(silu)
        bound = bound + dh @ np.abs(down[0]).T
    close(y, want, bound, 1.0, torch.bfloat16)


# ---- routing with experts that give no number -------------------------------------------

@pytest.mark.parametrize("e", [6, 70, 300])
def test_moe_experts_of_nan_logits_come_last(e):
    import torch
    rng = np.random.default_rng(e)
    n, d, f = 5, 64, 64
    gate, up, down = (_experts(rng, 6, f, d)[0] for _ in range(3))
    at = torch.arange(e, device="cuda") % 6
    part = lambda t: t.view(torch.uint8)[at].view(t.dtype)
    gate, up, down = (a._replace(values=part(a.values), meta=a.meta[at], scales=part(a.scales)) for a in (gate, up, down))
    x, _ = tensor(rng.standard_normal((n, d)), "bf16")
    r, _ = tensor(rng.standard_normal((e, d)), "bf16")
    y, ids, wts = sms.moe24_fp8(x, r, gate, up, down, 3, return_routing=True)
    sync()
    bad = [i for i in range(e) if i not in ids.unique().tolist()][:2]
    if e == 6 and len(bad) < 2:       # few experts: leave three of them numbers
        bad = [1, 2, 4]
    whole = r.clone()
    r[bad] = float("nan")
    y2, ids2, wts2 = sms.moe24_fp8(x, r, gate, up, down, 3, return_routing=True)
    sync()
    logits = f64(x) @ np.nan_to_num(f64(r)).T
    logits[:, bad] = -np.inf
    assert np.array_equal(ids2.cpu().numpy(), np.argsort(-logits, axis=1, kind="stable")[:, :3])
    assert bool(torch.isfinite(wts2).all()) and bool(torch.isfinite(y2).all())
    if e > 6:
        assert torch.equal(y2, y) and torch.equal(ids2, ids) and torch.equal(wts2, wts)
    # more chosen than there are numbers: the numbers first, then the lowest of the others
    keep, r = [0, 3], whole.clone()
    r[[i for i in range(e) if i not in keep]] = float("nan")
    _, ids3, wts3 = sms.moe24_fp8(x, r, gate, up, down, 4, return_routing=True)
    sync()
    order = np.argsort(-(f64(x) @ f64(whole).T)[:, keep], axis=1, kind="stable")
    assert np.array_equal(ids3[:, :2].cpu().numpy(), np.array(keep)[order])
    assert ids3[:, 2:].tolist() == [[1, 2]] * n
    assert bool(torch.isnan(wts3).all())
