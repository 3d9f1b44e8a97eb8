"""The binding of the 8-bit operators without a GPU: how its functions are called, and what it finds
out before a launch."""
import inspect

import pytest

import sparse_mask_search_amd as sms

torch = pytest.importorskip("torch")

ARGUMENTS = {
    "quant_fp8": ["X", "transpose", "stream"],
    "quant_fp8_both": ["X", "stream"],
    "compress24_fp8": ["W", "mask", "transpose", "stream"],
    "compress24_fp8_both": ["W", "mask", "stream"],
    "spmm24_fp8": ["X", "A", "out", "dtype", "stream"],
    "gemm_fp8": ["A", "B", "mask", "out", "dtype", "stream"],
    "moe24_fp8": ["x", "router", "gate", "up", "down", "topk", "out", "return_routing", "stream"],
}


@pytest.mark.parametrize("name", sorted(ARGUMENTS))
def test_arguments_have_names(name):
    """The signature names what a caller gives, and every argument may be given by its name."""
    fn = getattr(sms, name)
    params = inspect.signature(fn).parameters
    assert list(params) == ARGUMENTS[name]
    needed = [p for p in params.values() if p.default is inspect.Parameter.empty]
    with pytest.raises(TypeError, match="needs CUDA"):
        fn(**{p.name: torch.zeros(8, 128) for p in needed})
    with pytest.raises(TypeError, match=needed[0].name):
        fn()


def _refused(out, x):
    from sparse_mask_search_amd import _fp8
    try:
        _fp8._apart(out, x)
    except ValueError:
        return True
    return False


def test_outputs_over_operands_are_found():
    """Parts of operands are contiguous, of two dimensions or (stacked) three: they may lie before,
    behind or whole between two rows of a strided output."""
    buf = torch.zeros((6, 64), dtype=torch.bfloat16)
    flat = buf.view(-1)
    out = buf[1:5, :16]
    for first, size, over in ((0, 64, False), (0, 65, True), (64, 8, True), (80, 48, False), (79, 8, True),
                              (80, 49, True), (208, 48, False), (272, 64, False), (271, 8, True), (100, 100, True)):
        part = flat[first:first + size]
        assert _refused(out, part.view(1, size)) == over, (first, size)
        assert _refused(out, part.view(1, 1, size)) == over, (first, size)
        assert _refused(part.view(1, size), out) == over, (first, size)
    # several rows of an operand between two rows of the output, and over one
    assert not _refused(out, flat[144:176].view(4, 8))
    assert _refused(out, flat[144:200].view(7, 8))
    assert not _refused(out, flat[:0].view(1, 0))


def test_messages_name_the_arguments():
    from sparse_mask_search_amd import TsenorError
    assert "topk" in str(TsenorError(4, "tsenor_moe24_fp8"))
    assert "TSENOR_E4M3" in str(TsenorError(5, "tsenor_spmm24_fp8"))
    assert "tau" in str(TsenorError(4, "tsenor_mask"))


@pytest.mark.parametrize("name,args", [
    ("quant", dict(rows=1 << 32, cols=128, ld=128, vt=None, st=None)),
    ("quant", dict(rows=1 << 32, cols=1, ld=1)),
    ("compress", dict(batch=1 << 25, stride=4096, rows=4, cols=4, ld=4)),
    ("spmm", dict(n=1 << 20, m=1 << 20, ldy=1 << 20)),
    ("spmm", dict(n=1 << 35, m=8, ldy=8)),
    ("gemm", dict(p=1 << 20, q=1 << 20, k=1, ldc=1 << 20)),
    ("gemm", dict(p=1 << 32, q=60, k=0, ldc=64)),
])
def test_grids_of_the_largest_operands(name, args):
    """Operands of up to 2^40 entries whose workgroups do not fit one launch are refused on the host
    (no launch is made here: the pointers are not device memory)."""
    import test_fp8_abi as abi
    assert getattr(abi, name)(**args) == abi.SHAPE
