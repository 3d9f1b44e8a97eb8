"""GPU: bf16 tokens made to integers inside tsenor_gemm_int8, for every number that the entry point allows (the binding
asks for fewer), against numpy, bit for bit."""
import ctypes

import numpy as np
import pytest

import ops_ref as ref
import sparse_mask_search_amd as sms
from test_gpu_ops import _int8_operands, exactly, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", range(1, 17))
@pytest.mark.parametrize("m,k,pad", [(77, 200, 0), (16, 2048, 8), (300, 1001, 3)])
def test_tokens_inside_the_product(rows, m, k, pad):
    import torch
    say("tokens", rows, m, k, pad)
    assert rows * ref.pad(k) <= 32768
    rng = np.random.default_rng(rows * k)
    x = torch.from_numpy(rng.standard_normal((rows, k + pad)).astype(np.float32)).cuda().to(torch.bfloat16)[:, :k]
    if rows > 3:
        x[1], x[2, k // 2], x[3, 0] = 0, float("nan"), float("-inf")
    _, _, a = _int8_operands(rng, (), m, k)
    values, scales = ref.quant_int8(x.to(torch.float32).cpu().numpy())
    want = ref.gemm_int8(values, scales, a.values.cpu().numpy(), a.scales.cpu().numpy())
    for t, code in ((torch.bfloat16, sms.BF16), (torch.float32, sms.F32)):
        y = torch.full((rows + 1, m), 7.0, device="cuda", dtype=t)
        p = lambda v: ctypes.c_void_p(v.data_ptr())
        status = sms.lib().tsenor_gemm_int8(p(x), sms.BF16, None, rows, k + pad, p(a.values), p(a.scales), 1, m, k, None, p(y),
                                            code, m, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert status == 0
        exactly(y[:rows], want)
        assert bool((y[rows] == 7).all())
        exactly(sms.gemm_int8(x, a, dtype=t), want)
