"""GPU: the 8-bit operators where their numbers' range ends."""
import numpy as np
import pytest

import fp8_ref as ref
import sparse_mask_search_amd as sms
from test_gpu_fp8 import _experts, say, sync, tensor, words

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
