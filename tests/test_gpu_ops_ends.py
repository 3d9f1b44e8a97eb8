"""GPU: `ends` of the grouped operators at the ends of its type, through few rows, every tile and unaligned rows.
Small integers, compared bit for bit."""
import numpy as np
import pytest

import ops_ref as ref
import sparse_mask_search_amd as sms
from test_gpu_ops import _int8_operands, bf16, exactly, ints, say

pytestmark = pytest.mark.gpu

HIGH, LOW = 2 ** 31 - 1, -2 ** 31


@pytest.mark.parametrize("rows,m,k", [(10, 32, 64), (300, 96, 136), (300, 97, 45), (2900, 1000, 72), (3000, 2048, 72),
                                      (4100, 2560, 40)])
@pytest.mark.parametrize("ends", [[HIGH] * 3, [LOW] * 3, [LOW, 7, HIGH], [HIGH, LOW, 5], [LOW, LOW, HIGH], [5, HIGH, LOW]])
def test_ends_of_the_type(ends, rows, m, k):
    import torch
    say("ends", ends, rows, m, k)
    rng = np.random.default_rng(rows)
    e = torch.tensor(ends, dtype=torch.int32).cuda()
    assert e.tolist() == ends
    x, xv = bf16(ints(rng, (rows, k)))
    w, wv = bf16(ints(rng, (3, m, k)))
    dy, dyv = bf16(ints(rng, (rows, m)))
    exactly(sms.grouped_mm(x, w, e), ref.grouped_mm(xv, wv, ends, False)[0])
    exactly(sms.grouped_mm(dy, w, e, transpose=True), ref.grouped_mm(dyv, wv, ends, True)[0])
    exactly(sms.grouped_wgrad(dy, x, e), ref.grouped_wgrad(dyv, xv, ends)[0])
    qv, qs, q = _int8_operands(rng, (), rows, k)
    av, as_, a = _int8_operands(rng, (3,), m, k)
    want = np.zeros((rows, m), np.float32)
    for i, (first, end) in enumerate(ref.bounds(ends, rows)):
        want[first:end] = ref.gemm_int8(qv[first:end], qs[first:end], av[i], as_[i])
    exactly(sms.gemm_int8(q, a, ends=e, dtype=torch.float32), want)


def test_many_experts_at_the_ends_of_the_type():
    """Past 64 experts, whose scan takes 64 at a time: extremes on both sides of its borders."""
    import torch
    rng = np.random.default_rng(3)
    ends = rng.integers(0, 500, 200).tolist()
    for i in (0, 62, 63, 64, 65, 127, 128):
        ends[i] = LOW
    for last in (191, 199):
        some = list(ends)
        some[last] = HIGH
        e = torch.tensor(some, dtype=torch.int32).cuda()
        x, xv = bf16(ints(rng, (400, 40)))
        w, wv = bf16(ints(rng, (200, 72, 40)))
        dy, dyv = bf16(ints(rng, (400, 72)))
        exactly(sms.grouped_mm(x, w, e), ref.grouped_mm(xv, wv, some, False)[0])
        exactly(sms.grouped_mm(dy, w, e, transpose=True), ref.grouped_mm(dyv, wv, some, True)[0])
        exactly(sms.grouped_wgrad(dy, x, e), ref.grouped_wgrad(dyv, xv, some)[0])
