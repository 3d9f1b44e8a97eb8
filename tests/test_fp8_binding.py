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
