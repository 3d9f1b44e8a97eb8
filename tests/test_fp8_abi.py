"""C-ABI checks of the 8-bit operators that need no GPU: the library exports what
include/tsenor_fp8.h declares and refuses invalid arguments before any HIP call."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import fp8_ref as ref
import sparse_mask_search_amd as sms

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tsenor_fp8.h")
FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1008)  # not 16-byte aligned
OK, NULL, SHAPE, NM, PARAM, DTYPE, HIP = range(7)


def test_exports_every_declared_symbol():
    names = sorted(set(re.findall(r"^(?:int|size_t)\s+(tsenor_\w+)\s*\(", open(HEADER).read(), re.M)))
    assert names == ["tsenor_compress24_fp8", "tsenor_gemm_fp8", "tsenor_moe24_fp8",
                     "tsenor_moe24_fp8_workspace", "tsenor_quant_fp8", "tsenor_spmm24_fp8"]
    out = subprocess.check_output(["nm", "-D", "--defined-only", sms.library_path()], text=True)
    exported = set(re.findall(r"\bT (tsenor_\w+)", out))
    assert set(names) <= exported


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "tsenor_fp8.h"\nint main(void) { return TSENOR_E4M3 != 2; }\n')
    subprocess.check_call(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src),
                           "-o", str(tmp_path / "t.o")])


def quant(X=FAKE, dt=1, rows=8, cols=64, ld=64, v=FAKE, s=FAKE, vt=FAKE, st=FAKE):
    return sms.lib().tsenor_quant_fp8(X, dt, rows, cols, ld, v, s, vt, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), NULL), (dict(v=None), NULL), (dict(st=None), NULL),
    (dict(v=None, s=None, vt=None, st=None), NULL), (dict(dt=2), DTYPE), (dict(dt=-1), DTYPE),
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(ld=63), SHAPE), (dict(v=ODD), SHAPE),
    (dict(vt=ODD), SHAPE), (dict(X=ctypes.c_void_p(0x1001)), SHAPE),
    (dict(rows=1 << 60), SHAPE), (dict(cols=1 << 60, ld=1 << 60), SHAPE), (dict(rows=0), OK),
])
def test_quant_rejects(kw, code):
    assert quant(**kw) == code


def compress(W=FAKE, dt=1, batch=2, stride=64 * 64, rows=64, cols=64, ld=64, mask=FAKE, v=FAKE, m=FAKE,
             s=FAKE, vt=FAKE, mt=FAKE, st=FAKE):
    return sms.lib().tsenor_compress24_fp8(W, dt, batch, stride, rows, cols, ld, mask, v, m, s, vt, mt, st,
                                           None, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(W=None), NULL), (dict(mask=None), NULL), (dict(m=None), NULL), (dict(st=None), NULL),
    (dict(v=None, m=None, s=None, vt=None, mt=None, st=None), NULL), (dict(dt=2), DTYPE),
    (dict(rows=62), SHAPE), (dict(cols=62), SHAPE), (dict(ld=60), SHAPE), (dict(rows=0), SHAPE),
    (dict(batch=-1), SHAPE), (dict(stride=4000), SHAPE), (dict(v=ODD), SHAPE), (dict(mt=ODD), SHAPE),
    (dict(batch=1 << 50), SHAPE), (dict(rows=1 << 40), SHAPE), (dict(batch=0), OK),
])
def test_compress_rejects(kw, code):
    assert compress(**kw) == code


def spmm(X=FAKE, xt=2, xs=FAKE, n=20, ldx=128, v=FAKE, me=FAKE, s=FAKE, m=64, k=100, Y=FAKE, yt=1, ldy=64):
    return sms.lib().tsenor_spmm24_fp8(X, xt, xs, n, ldx, v, me, s, m, k, Y, yt, ldy, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), NULL), (dict(xs=None), NULL), (dict(v=None), NULL), (dict(me=None), NULL),
    (dict(s=None), NULL), (dict(Y=None), NULL), (dict(xt=0), DTYPE), (dict(xt=3), DTYPE), (dict(yt=2), DTYPE),
    (dict(n=-1), SHAPE), (dict(m=0), SHAPE), (dict(k=0), SHAPE), (dict(ldx=112), SHAPE), (dict(ldx=136), SHAPE),
    (dict(ldy=63), SHAPE), (dict(X=ODD), SHAPE), (dict(v=ODD), SHAPE), (dict(me=ODD), SHAPE),
    (dict(Y=ctypes.c_void_p(0x1001)), SHAPE), (dict(xt=1, xs=None, n=17), SHAPE), (dict(m=1 << 60, ldy=1 << 60), SHAPE),
    (dict(xt=1, xs=None, n=16, ldx=99), SHAPE), (dict(n=0, X=None, Y=None), OK),
])
def test_spmm_rejects(kw, code):
    assert spmm(**kw) == code


def gemm(A=FAKE, sa=FAKE, p=8, B=FAKE, sb=FAKE, q=40, k=100, mask=FAKE, C=FAKE, ct=1, ldc=40):
    return sms.lib().tsenor_gemm_fp8(A, sa, p, B, sb, q, k, mask, C, ct, ldc, None)


@pytest.mark.parametrize("kw,code", [
    (dict(A=None), NULL), (dict(sa=None), NULL), (dict(B=None), NULL), (dict(sb=None), NULL),
    (dict(C=None), NULL), (dict(ct=2), DTYPE), (dict(p=0), SHAPE), (dict(q=-3), SHAPE), (dict(k=-1), SHAPE),
    (dict(ldc=39), SHAPE), (dict(A=ODD), SHAPE), (dict(B=ODD), SHAPE), (dict(mask=ctypes.c_void_p(0x1002)), SHAPE),
    (dict(p=1 << 60), SHAPE),
])
def test_gemm_rejects(kw, code):
    assert gemm(**kw) == code


def moe(X=FAKE, n=4, ldx=64, d=64, r=FAKE, ldr=64, e=8, topk=2, gv=FAKE, gm=FAKE, gs=FAKE, dv=FAKE, f=32, ws=FAKE,
        size=1 << 30, Y=FAKE, ldy=64):
    return sms.lib().tsenor_moe24_fp8(X, n, ldx, d, r, ldr, e, topk, gv, gm, gs, FAKE, FAKE, FAKE, dv, FAKE, FAKE,
                                      f, ws, size, Y, ldy, None, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), NULL), (dict(r=None), NULL), (dict(gv=None), NULL), (dict(gs=None), NULL),
    (dict(ws=None), NULL), (dict(Y=None), NULL), (dict(topk=0), PARAM), (dict(topk=9), PARAM),
    (dict(topk=17, e=32), PARAM), (dict(e=513), PARAM), (dict(e=0), PARAM), (dict(n=65), SHAPE), (dict(n=-1), SHAPE),
    (dict(d=0), SHAPE), (dict(f=0), SHAPE), (dict(ldx=63), SHAPE), (dict(ldr=63), SHAPE), (dict(ldy=63), SHAPE),
    (dict(gv=ODD), SHAPE), (dict(gm=ODD), SHAPE), (dict(ws=ODD), SHAPE), (dict(size=100), SHAPE),
    (dict(n=0, X=None, Y=None, ws=None), OK),
])
def test_moe_rejects(kw, code):
    assert moe(**kw) == code


HUGE = (1 << 63) - 1


@pytest.mark.parametrize("call,kw", [
    (quant, dict(rows=HUGE)), (quant, dict(cols=HUGE, ld=HUGE)), (quant, dict(ld=HUGE)), (quant, dict(rows=HUGE, cols=1)),
    (compress, dict(batch=HUGE)), (compress, dict(rows=HUGE - 3)), (compress, dict(cols=HUGE - 3, ld=HUGE)),
    (compress, dict(stride=HUGE)), (spmm, dict(n=HUGE)), (spmm, dict(m=HUGE, ldy=HUGE)), (spmm, dict(k=HUGE)),
    (spmm, dict(ldy=HUGE)), (spmm, dict(k=HUGE, ldx=HUGE - 15)), (gemm, dict(p=HUGE)), (gemm, dict(q=HUGE, ldc=HUGE)),
    (gemm, dict(k=HUGE)), (gemm, dict(ldc=HUGE)), (moe, dict(d=HUGE, ldx=HUGE, ldr=HUGE, ldy=HUGE)), (moe, dict(f=HUGE)),
    (moe, dict(ldx=HUGE)), (moe, dict(ldr=HUGE)), (moe, dict(ldy=HUGE)),
])
def test_sums_of_sizes_do_not_wrap(call, kw):
    assert call(**kw) == SHAPE


@pytest.mark.parametrize("call,kw", [
    (quant, dict(rows=1 << 28, cols=129, ld=129, vt=None, st=None)),     # 2^25 workgroups of 256 threads
    (quant, dict(rows=1 << 31, cols=129, ld=129)),                       # 2^25 tiles
    (compress, dict(batch=1 << 24, stride=4096)),
    (spmm, dict(n=1, m=1 << 28, k=64, ldy=1 << 28)),                     # 2^24 workgroups of 512 threads
    (gemm, dict(p=1 << 31, q=40, k=1)),
    (moe, dict(n=64, e=512, topk=8, f=1 << 20, size=1 << 40)),           # 2^24 workgroups of 256 threads
])
def test_grids_past_a_launch_are_refused(call, kw):
    assert call(**kw) == SHAPE


def test_moe_workspace():
    w = sms.lib().tsenor_moe24_fp8_workspace
    assert w(4, 64, 32, 8, 2) >= 4 * 8 * 8 + 4 * 128 * 2 + 8 * 128 * 2 + 8 * 4
    assert w(65, 64, 32, 8, 2) == 0 and w(4, 64, 32, 8, 9) == 0
    need = w(4, 64, 32, 8, 2)
    assert moe(size=need - 1) == SHAPE


def test_binding_requires_device_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(8, 128)
    a = sms.DenseFp8(x.to(torch.float8_e4m3fn), x, 128)
    for call in (lambda: sms.quant_fp8(x), lambda: sms.quant_fp8_both(x),
                 lambda: sms.compress24_fp8(x, x), lambda: sms.spmm24_fp8(x, a),
                 lambda: sms.gemm_fp8(a, a), lambda: sms.moe24_fp8(x, x, a, a, a, 1)):
        with pytest.raises(TypeError):
            call()


def test_reference_rounding():
    """The tests' own e4m3 rounding: codes round-trip, ties go to even codes, the border of
    the scale is inclusive."""
    finite = [b for b in range(256) if (b & 0x7F) != 0x7F]
    assert np.array_equal(ref.round_e4m3(ref.E4M3[finite]), np.array(finite, np.uint8))
    assert ref.E4M3[0x7E] == 448.0 and ref.E4M3[1] == 2.0 ** -9
    assert ref.round_e4m3(np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == [
        ref.round_e4m3(np.array([16.0]))[0], ref.round_e4m3(np.array([20.0]))[0], 0, 2]
    assert ref.exponent(np.array([448.0, 448.0001, 0.0, 1e-45, 3.3e38])).tolist() == [0, 1, 0, -127, 120]


@pytest.mark.parametrize("x,out,fine", [
    (np.s_[0:4, 0:32], np.s_[0:4, 32:64], True),     # side by side in one buffer
    (np.s_[0:4, 32:64], np.s_[0:4, 0:32], True),
    (np.s_[0:4, :], np.s_[4:8, :], True),            # one above the other
    (np.s_[2:3, 0:8], np.s_[0:8, 8:64], True),       # one row beside many
    (np.s_[0:4, 0:32], np.s_[0:4, 0:32], False),
    (np.s_[0:4, 0:33], np.s_[0:4, 32:64], False),
    (np.s_[0:4, 31:64], np.s_[0:4, 0:32], False),
    (np.s_[0:4, :], np.s_[3:7, :], False),
    (np.s_[2:3, 0:9], np.s_[0:8, 8:64], False),
    (np.s_[0:0, :], np.s_[0:0, :], True),
])
def test_outputs_over_inputs_are_found(x, out, fine):
    import torch
    from sparse_mask_search_amd import _fp8
    buf = torch.zeros((8, 64), dtype=torch.bfloat16)
    if fine:
        _fp8._apart(buf[out], buf[x])
    else:
        with pytest.raises(ValueError, match="overlaps"):
            _fp8._apart(buf[out], buf[x])
    _fp8._apart(torch.zeros((8, 64)), buf)


def test_outputs_over_inputs_of_another_width():
    import torch
    from sparse_mask_search_amd import _fp8
    buf = torch.zeros((4, 64), dtype=torch.float32)
    halves = buf.view(torch.bfloat16)  # the same rows, 128 entries each
    _fp8._apart(buf[:, 32:], halves[:, :64])
    with pytest.raises(ValueError, match="overlaps"):
        _fp8._apart(buf[:, 31:], halves[:, :64])
    with pytest.raises(ValueError, match="overlaps"):
        _fp8._apart(buf.view(8, 32), halves[:, :64])  # other rows over the same bytes
