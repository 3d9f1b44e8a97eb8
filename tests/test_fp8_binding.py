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
