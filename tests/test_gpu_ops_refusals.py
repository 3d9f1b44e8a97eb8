"""GPU: what the binding of include/tsenor_ops.h refuses by itself, on device tensors: the error's type and its message
name the argument, the library is not called and no argument is written."""
import pytest

import sparse_mask_search_amd as sms

pytestmark = pytest.mark.gpu


def tensors(v):
    import torch
    if isinstance(v, torch.Tensor):
        yield v
    elif isinstance(v, (list, tuple, dict)):
        for u in (v.values() if isinstance(v, dict) else v):
            yield from tensors(u)


def test_refused_by_the_binding(monkeypatch):
    import torch

    import ops_refusals
    from sparse_mask_search_amd import _ops
    calls = ops_refusals.calls("cuda", sms)
    x, w = torch.zeros(40, 32, device="cuda", dtype=torch.bfloat16), torch.zeros(4, 64, 32, device="cuda", dtype=torch.bfloat16)
    ends, a = torch.zeros(4, device="cuda", dtype=torch.int32), sms.quant_int8(w[0])
    calls += [
        ("ends on the host", "grouped_mm", (x, w, ends.cpu()), {}, ValueError, "ends must be"),
        ("W on the host", "grouped_mm", (x, w.cpu(), ends), {}, TypeError, "W must be a CUDA"),
        ("X on the host", "grouped_mm", (x.cpu(), w, ends), {}, TypeError, "needs CUDA"),
        ("out on the host", "grouped_mm", (x, w, ends), dict(out=torch.zeros(40, 64, dtype=torch.bfloat16)), TypeError, "out must be a CUDA"),
        ("scales on the host", "gemm_int8", (x, a._replace(scales=a.scales.cpu())), {}, ValueError, "A.scales must be a contiguous"),
        ("no gradients", "clip_grads", ([], 1.0), {}, TypeError, "needs CUDA"),
        ("gradients by a generator", "grad_norm", (t for t in [x]), {}, TypeError, "needs CUDA"),
        ("a gradient on the host", "clip_grads", ([x, x.cpu()], 1.0), {}, TypeError, r"grads\[1\] must be a tensor on"),
    ]
    torch.cuda.synchronize()
    monkeypatch.setattr(_ops, "lib", lambda: pytest.fail("the library was called"))
    for name, fn, args, named, error, message in calls:
        print("[refused]", fn, name, flush=True)
        if not isinstance(args, tuple):
            args = (args,)
        with pytest.raises(error, match=message) as found:
            getattr(sms, fn)(*args, **named)
        assert found.type is error
    assert all(bool((t == 0).all()) for c in calls for t in tensors([c[2], c[3]]) if t is not a.values and t is not a.scales)


def test_refused_by_the_library():
    """What the binding leaves to the library's own checks."""
    import torch
    x, w = torch.zeros(40, 32, device="cuda", dtype=torch.bfloat16), torch.zeros(4, 64, 32, device="cuda", dtype=torch.bfloat16)
    ends, g = torch.zeros(4, device="cuda", dtype=torch.int32), torch.zeros(4, 40, device="cuda")
    values = torch.zeros(64 * 128 + 1, device="cuda", dtype=torch.int8)[1:].view(64, 128)
    many = torch.zeros(1025, device="cuda", dtype=torch.int32)
    for name, call, message in (
            ("experts past 1024", lambda: sms.grouped_mm(x, w[:1].expand(1025, -1, -1), many), "parameter"),
            ("weights of one place", lambda: sms.grouped_mm(x, w[:1].expand(4, -1, -1), ends), "shape"),
            ("k past 2^17", lambda: sms.quant_int8(torch.zeros(1, (1 << 17) + 1, device="cuda")), "shape"),
            ("unaligned integers", lambda: sms.gemm_int8(x, sms.DenseInt8(values, torch.zeros(64, device="cuda"), 32)), "alignment"),
            ("a negative limit", lambda: sms.clip_grads([g], -1.0), "parameter"),
            ("a NaN limit", lambda: sms.clip_grads([g], float("nan")), "parameter")):
        print("[refused]", name, flush=True)
        with pytest.raises(sms.TsenorError, match=message):
            call()
