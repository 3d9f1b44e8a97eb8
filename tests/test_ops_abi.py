"""C-ABI and binding checks of the operators of include/tsenor_ops.h that need no GPU: exports, names,
and invalid arguments refused before any HIP call."""
import ctypes
import inspect
import os
import re
import subprocess

import pytest

import sparse_mask_search_amd as sms

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tsenor_ops.h")
FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1001)
EIGHT = ctypes.c_void_p(0x1008)
OK, NULL, SHAPE, NM, PARAM, DTYPE, HIP = range(7)


def test_exports_every_declared_symbol():
    names = sorted(set(re.findall(r"^(?:int|size_t)\s+(tsenor_\w+)\s*\(", open(HEADER).read(), re.M)))
    assert names == ["tsenor_clip_grads", "tsenor_gemm_int8", "tsenor_grad_norm", "tsenor_grads_workspace",
                     "tsenor_grouped_mm", "tsenor_grouped_wgrad", "tsenor_quant_int8"]
    out = subprocess.check_output(["nm", "-D", "--defined-only", sms.library_path()], text=True)
    assert set(names) <= set(re.findall(r"\bT (tsenor_\w+)", out))


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "tsenor_ops.h"\n#include "tsenor_fp8.h"\n'
                   "int main(void) { return TSENOR_INT8 != 3 || sizeof(tsenor_grad) != 64; }\n")
    exe = str(tmp_path / "t")
    subprocess.check_call(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe])
    subprocess.check_call([exe])


def mm(X=FAKE, rows=20, ldx=64, W=FAKE, tr=0, experts=4, stride=96 * 64, ldw=64, m=96, k=64, ends=FAKE, Y=FAKE, yt=1,
       ldy=96):
    return sms.lib().tsenor_grouped_mm(X, rows, ldx, W, tr, experts, stride, ldw, m, k, ends, Y, yt, ldy, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), NULL), (dict(W=None), NULL), (dict(ends=None), NULL), (dict(Y=None), NULL), (dict(yt=2), DTYPE),
    (dict(tr=2), PARAM), (dict(tr=-1), PARAM), (dict(experts=0), PARAM), (dict(experts=1025, stride=0), PARAM),
    (dict(rows=-1), SHAPE), (dict(rows=1 << 30), SHAPE), (dict(m=0), SHAPE), (dict(k=0), SHAPE), (dict(ldx=63), SHAPE),
    (dict(k=1 << 30, ldx=1 << 30, ldw=1 << 30, stride=1 << 37, rows=1), SHAPE), (dict(ldw=63), SHAPE),
    (dict(ldy=95), SHAPE), (dict(stride=96 * 64 - 1), SHAPE), (dict(tr=1, ldw=95), SHAPE),
    (dict(X=ODD), SHAPE), (dict(W=ODD), SHAPE), (dict(ends=ctypes.c_void_p(0x1002)), SHAPE), (dict(Y=ODD), SHAPE),
    (dict(yt=0, Y=ctypes.c_void_p(0x1002)), SHAPE), (dict(k=1 << 41, ldx=1 << 41, ldw=1 << 41), SHAPE),
    (dict(rows=(1 << 31) - 1, ldx=1 << 30, stride=1 << 62), SHAPE), (dict(rows=0, X=None, Y=None), OK),
    (dict(rows=(1 << 31) - 1, m=1 << 9, ldy=1 << 9, stride=1 << 20), SHAPE), (dict(stride=1 << 40), SHAPE),
])
def test_grouped_mm_rejects(kw, code):
    assert mm(**kw) == code


def wgrad(dY=FAKE, lddy=96, X=FAKE, ldx=64, rows=20, experts=4, m=96, k=64, ends=FAKE, mask=FAKE, C=FAKE, ct=1,
          stride=96 * 64, ldc=64):
    return sms.lib().tsenor_grouped_wgrad(dY, lddy, X, ldx, rows, experts, m, k, ends, mask, C, ct, stride, ldc, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), NULL), (dict(dY=None), NULL), (dict(ends=None), NULL), (dict(C=None), NULL), (dict(ct=2), DTYPE),
    (dict(experts=0), PARAM), (dict(experts=2000), PARAM), (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE),
    (dict(m=0), SHAPE), (dict(k=0), SHAPE), (dict(lddy=95), SHAPE), (dict(ldx=63), SHAPE), (dict(ldc=63), SHAPE),
    (dict(stride=96 * 64 - 1), SHAPE), (dict(X=ODD), SHAPE), (dict(dY=ODD), SHAPE), (dict(C=ODD), SHAPE),
    (dict(mask=ctypes.c_void_p(0x1002)), SHAPE), (dict(m=1 << 20, lddy=1 << 20, ldc=1 << 20, k=1 << 20, ldx=1 << 20,
                                                       stride=1 << 40), SHAPE),
])
def test_grouped_wgrad_rejects(kw, code):
    assert wgrad(**kw) == code


def quant(X=FAKE, dt=1, batch=2, stride=640, rows=10, cols=64, ldx=64, v=FAKE, s=FAKE):
    return sms.lib().tsenor_quant_int8(X, dt, batch, stride, rows, cols, ldx, v, s, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), NULL), (dict(v=None), NULL), (dict(s=None), NULL), (dict(dt=2), DTYPE), (dict(batch=-1), SHAPE),
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=(1 << 17) + 1, ldx=1 << 18), SHAPE), (dict(ldx=63), SHAPE),
    (dict(stride=639), SHAPE), (dict(X=ODD), SHAPE), (dict(v=EIGHT), SHAPE), (dict(s=ctypes.c_void_p(0x1002)), SHAPE),
    (dict(rows=0, X=None, v=None, s=None), OK), (dict(batch=0), OK), (dict(rows=1 << 38, stride=1 << 39), SHAPE),
    (dict(batch=1, rows=1 << 36, cols=1, ldx=1), SHAPE),
])
def test_quant_int8_rejects(kw, code):
    assert quant(**kw) == code


def gemm(X=FAKE, xt=3, xs=FAKE, rows=20, ldx=128, A=FAKE, as_=FAKE, experts=4, m=96, k=100, ends=FAKE, Y=FAKE, yt=1,
         ldy=96):
    return sms.lib().tsenor_gemm_int8(X, xt, xs, rows, ldx, A, as_, experts, m, k, ends, Y, yt, ldy, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), NULL), (dict(xs=None), NULL), (dict(A=None), NULL), (dict(as_=None), NULL), (dict(Y=None), NULL),
    (dict(xt=2), DTYPE), (dict(xt=0), DTYPE), (dict(yt=3), DTYPE), (dict(experts=0), PARAM), (dict(ends=None), PARAM),
    (dict(experts=1025), PARAM), (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(m=0), SHAPE),
    (dict(k=0), SHAPE), (dict(k=(1 << 17) + 1, ldx=(1 << 17) + 128), SHAPE), (dict(ldx=256), SHAPE), (dict(ldy=95), SHAPE),
    (dict(X=EIGHT), SHAPE), (dict(A=EIGHT), SHAPE), (dict(Y=ODD), SHAPE), (dict(m=1 << 39, ldy=1 << 39), SHAPE),
    (dict(xt=1, xs=None, ldx=100), SHAPE),                                     # bf16 tokens: no groups,
    (dict(xt=1, xs=None, ldx=100, experts=1, ends=None, rows=17), SHAPE),      # at most 16
    (dict(xt=1, xs=None, ldx=99, experts=1, ends=None, rows=16), SHAPE),
    (dict(xt=1, xs=None, ldx=100, experts=1, ends=None, X=ODD, rows=16), SHAPE),
    (dict(m=1 << 30, ldy=1 << 30, experts=1), SHAPE), (dict(rows=1 << 30), SHAPE),
    (dict(rows=0, X=None, Y=None, xs=None), OK),
])
def test_gemm_int8_rejects(kw, code):
    assert gemm(**kw) == code


def clip(n=1, count=None, max_norm=1.0, work=FAKE, size=None, norm=FAKE, write=True, grads=True, **kw):
    one = dict(grad=0x1000, out=0x2000, mask=0, dtype=0, rows=4, cols=8, ld=8, ldo=8)
    one.update(kw)
    table = (ctypes.c_int64 * (8 * n))(*(list(one.values()) * n))
    count = n if count is None else count
    size = sms.lib().tsenor_grads_workspace(max(count, 0)) if size is None else size
    p = ctypes.cast(table, ctypes.c_void_p) if grads else None
    if write:
        return sms.lib().tsenor_clip_grads(p, count, max_norm, work, size, norm, None)
    return sms.lib().tsenor_grad_norm(p, count, work, size, norm, None)


@pytest.mark.parametrize("kw,code", [
    (dict(grads=False), NULL), (dict(work=None), NULL), (dict(norm=None), NULL), (dict(grad=0), NULL), (dict(out=0), NULL),
    (dict(count=-1), PARAM), (dict(max_norm=-1.0), PARAM), (dict(max_norm=float("nan")), PARAM), (dict(dtype=2), DTYPE),
    (dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE), (dict(ld=7), SHAPE), (dict(ldo=7), SHAPE), (dict(grad=0x1002), SHAPE),
    (dict(out=0x2001), SHAPE), (dict(mask=0x3002), SHAPE), (dict(out=0x1000, ldo=9), SHAPE), (dict(size=100), SHAPE),
    (dict(work=ctypes.c_void_p(0x1004)), SHAPE), (dict(rows=1 << 40), SHAPE), (dict(n=3, dtype=7), DTYPE),
    (dict(write=False, grad=0), NULL), (dict(write=False, count=-3), PARAM), (dict(write=False, size=0), SHAPE),
])
def test_clip_rejects(kw, code):
    assert clip(**kw) == code


def test_workspace_grows_with_the_list():
    size = sms.lib().tsenor_grads_workspace
    assert 0 < size(0) <= size(1) <= size(100) < size(10000) < 1 << 22


ARGUMENTS = {
    "grouped_mm": ["X", "W", "ends", "transpose", "out", "dtype", "stream"],
    "grouped_wgrad": ["dY", "X", "ends", "mask", "out", "dtype", "stream"],
    "quant_int8": ["X", "stream"],
    "gemm_int8": ["X", "A", "ends", "out", "dtype", "stream"],
    "grad_norm": ["grads", "masks", "stream"],
    "clip_grads": ["grads", "max_norm", "masks", "out", "stream"],
}


@pytest.mark.parametrize("name", sorted(ARGUMENTS))
def test_arguments_have_names(name):
    fn = getattr(sms, name)
    params = inspect.signature(fn).parameters
    assert list(params) == ARGUMENTS[name]
    needed = [p for p in params.values() if p.default is inspect.Parameter.empty]
    with pytest.raises(TypeError, match="needs CUDA"):
        fn(**{p.name: torch.zeros(8, 128) for p in needed})
    with pytest.raises(TypeError, match=needed[0].name):
        fn()


def test_lists_that_overlap_are_found():
    from sparse_mask_search_amd import _ops
    buf = torch.zeros(8, 64)
    a, b = buf[:, :32], buf[:, 32:]

    def check(grads, masks=None, out=None):
        _ops._grad_list(torch, grads, masks, out, True)
    words = buf.view(torch.int32)
    check([a, b])
    check([buf[:4], buf[4:]])
    check([buf[:4]], [words[4:6].view(-1)[:8].view(4, 2)])
    check([a.t(), b.t()])
    check([buf[:0], buf])
    check([buf[:2]], out=[buf[2:4]])
    check([a[:4], b[:4]], out=[a[4:], b[4:]])
    _ops._grad_list(torch, [buf, buf], None, None, False)  # a norm writes nothing
    for grads, masks, out in (([buf, buf], None, None), ([a, buf[:, 31:40]], None, None), ([buf[:5], buf[4:]], None, None),
                              ([buf[:4]], None, [buf[2:6]]), ([buf[:2], buf[2:4]], None, [buf[4:6], buf[5:7]]),
                              ([buf[:2], buf[2:4]], None, [buf[4:6], buf[:2]]),
                              ([buf[:4]], [words[1:2].view(-1)[:8].view(4, 2)], None)):
        with pytest.raises(ValueError, match="overlaps"):
            check(grads, masks, out)


def test_gradients_that_do_not_fit_are_refused():
    from sparse_mask_search_amd import _ops
    g, m = torch.zeros(4, 40), torch.zeros(4, 2, dtype=torch.int32)
    ok = ([g], [m], [torch.zeros(4, 40)])
    _ops._grad_list(torch, *ok, True)
    for change, match in ((dict(grads=[g.double()]), "grads"), (dict(masks=[m, m]), "masks"), (dict(masks=[m.long()]), "masks"),
                          (dict(masks=[m[:, :1]]), "masks"), (dict(masks=[m[:2]]), "masks"), (dict(out=[]), "out"),
                          (dict(out=[g[:2]]), "out"), (dict(out=[torch.zeros(4, 40, dtype=torch.bfloat16)]), "out"),
                          (dict(grads=[torch.zeros(4, 4, 80)[..., ::2]], masks=None, out=None), "grads"),
                          (dict(grads=[torch.zeros(40, 4).t()], out=None), "grads"), (dict(grads=(x for x in [g])), "grads"),
                          (dict(grads=[torch.zeros(())], masks=[m], out=None), "masks"), (dict(grads=[None]), "device")):
        args = dict(grads=[g], masks=[m], out=None)
        args.update(change)
        with pytest.raises((TypeError, ValueError, AttributeError), match=match):
            _ops._grad_list(torch, args["grads"], args["masks"], args["out"], True)
