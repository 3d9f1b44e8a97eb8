"""GPU: every kernel that a product of include/tsenor_ops.h can take, against numpy in 64 bits, bit for bit:
small integers, whose products and sums are exact in fp32 (below 2^24), so that only the output type rounds;
8-bit integers with their scales in the order that the header gives.  tests/test_ops_forms.py asserts that
these sizes reach each kernel, with reductions longer than its ring and more tiles than workgroups."""
import numpy as np
import pytest

import ops_ref as ref
import ops_sizes as sizes
import sparse_mask_search_amd as sms
from test_gpu_ops import _int8_operands, ends_of, say, torch_type, words

pytestmark = pytest.mark.gpu


def operand(rng, shape):
    """A bf16 tensor of small integers and their values."""
    import torch
    v = rng.integers(-3, 4, shape, dtype=np.int8)
    return torch.from_numpy(v).cuda().to(torch.bfloat16), v.astype(np.float64)


def same(got, want):
    import torch
    want = torch.from_numpy(want.astype(np.float32)).to(got.dtype).cuda()
    assert got.shape == want.shape
    wrong = got != want
    assert not bool(wrong.any()), (int(wrong.sum()), wrong.nonzero()[:4].tolist())


@pytest.mark.parametrize("op", ["product", "transposed", "integers"])
@pytest.mark.parametrize("case", sizes.PRODUCTS, ids=lambda c: "-".join(map(str, c[:5])))
def test_products(case, op):
    import torch
    rows, experts, m, k = case[:4]
    say(op, *case)
    counts = sizes.counts_of(rows, experts)
    rng = np.random.default_rng(rows + m)
    if op == "integers":
        xv, xs, x = _int8_operands(rng, (), rows, k)
        av, as_, a = _int8_operands(rng, (experts,), m, k)
        want = np.zeros((rows, m), np.float32)
        for e, (i, j) in enumerate(ref.bounds(np.cumsum(counts), rows)):
            sums = xv[i:j].astype(np.float64) @ av[e].astype(np.float64).T  # exact: below 2^53
            want[i:j] = sums.astype(np.float32) * xs[i:j, None] * as_[e][None]
        for t in (torch.bfloat16, torch.float32):
            same(sms.gemm_int8(x, a, ends=ends_of(counts), dtype=t), want)
        return
    turn = op == "transposed"
    x, xv = operand(rng, (rows, k))
    w, wv = operand(rng, (experts, k, m) if turn else (experts, m, k))
    want, _ = ref.grouped_mm(xv, wv, np.cumsum(counts), turn)
    for t in (torch.bfloat16, torch.float32):
        same(sms.grouped_mm(x, w, ends_of(counts), transpose=turn, dtype=t), want)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("case", sizes.GRADIENTS, ids=lambda c: "-".join(map(str, c)))
def test_gradients(case, masked):
    rows, experts, m, k = case[:4]
    say("gradient", *case, masked)
    counts = sizes.counts_of(rows, experts)
    rng = np.random.default_rng(rows + k)
    x, xv = operand(rng, (rows, k))
    dy, dyv = operand(rng, (rows, m))
    keep = rng.random((experts, m, k), dtype=np.float32) < 0.5 if masked else None
    want, _ = ref.grouped_wgrad(dyv, xv, np.cumsum(counts), keep)
    for name in ("bf16", "f32"):
        same(sms.grouped_wgrad(dy, x, ends_of(counts), mask=words(keep) if masked else None, dtype=torch_type(name)), want)
