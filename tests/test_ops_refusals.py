"""What the binding of include/tsenor_ops.h refuses by itself, without a GPU: the error's type and its message name the
argument, and the library is not called.  (Its tests of memory that a GPU can see are left out here.)"""
import pytest

import sparse_mask_search_amd as sms

torch = pytest.importorskip("torch")

import ops_refusals  # noqa: E402

CALLS = ops_refusals.calls("cpu", sms)


@pytest.fixture()
def host_only(monkeypatch):
    from sparse_mask_search_amd import _ops

    def matrix(torch, t, name, dim=2):
        if t.dim() != dim or (t.stride(-1) != 1 and t.shape[-1] > 1):
            raise ValueError(f"{name} must be {dim}-D with unit column stride")
    monkeypatch.setattr(_ops, "_matrix", matrix)
    monkeypatch.setattr(_ops, "lib", lambda: pytest.fail("the library was called"))


@pytest.mark.parametrize("call", CALLS, ids=lambda c: f"{c[1]}: {c[0]}")
def test_refused_by_the_binding(call, host_only):
    _, fn, args, named, error, message = call
    with pytest.raises(error, match=message) as found:
        getattr(sms, fn).__wrapped__(torch, *args, **named)
    assert found.type is error


def test_what_is_allowed_reaches_the_library(monkeypatch, host_only):
    """The operands that the refused calls are made of pass by themselves."""
    from sparse_mask_search_amd import _ops

    class Reached(Exception):
        pass

    def lib():
        raise Reached
    monkeypatch.setattr(_ops, "lib", lib)
    x, w, ends = CALLS[1][2][0].new_zeros(40, 32), CALLS[1][2][1], CALLS[1][2][2]
    dy, a = x.new_zeros(40, 64), next(c for c in CALLS if c[0] == "A no stack with ends")[2][1]
    for fn, args, named in (("grouped_mm", (x, w, ends), {}), ("grouped_mm", (dy, w, ends), dict(transpose=True)),
                            ("grouped_mm", (x, w, ends), dict(out=dy)), ("grouped_wgrad", (dy, x, ends), {}),
                            ("quant_int8", (x,), {}), ("gemm_int8", (x, a), dict(out=dy)), ("clip_grads", ([x, dy], 1.0), {}),
                            ("grad_norm", ([x, x],), {})):
        with pytest.raises(Reached):
            getattr(sms, fn).__wrapped__(torch, *args, **named)
