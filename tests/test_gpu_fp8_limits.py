"""GPU: the 8-bit operators where their numbers' range ends."""
import numpy as np
import pytest

import sparse_mask_search_amd as sms
from test_gpu_fp8 import _experts, say, sync

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
