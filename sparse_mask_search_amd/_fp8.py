"""Binding of the 8-bit operators (include/tsenor_fp8.h).

Operands are named tuples of torch tensors: ``DenseFp8`` (activations,
gradients: blocks of 1 x 128) and ``Sparse24Fp8`` (weights under a 2:4 mask:
blocks of 128 x 128, also stacked, one operand per expert).  Values are
float8_e4m3fn, scales float8_e8m0fnu (powers of two), rows are padded with
zeros to a multiple of 128.  With ``stream`` a call runs on that stream and
takes its memory there; otherwise it runs on the current stream of the
tensors' device.
"""
from __future__ import annotations

import functools
import inspect
from typing import NamedTuple

from . import _lib
from ._lib import BF16, F32, TsenorError, lib

E4M3 = 2


class DenseFp8(NamedTuple):
    """Dense operand [rows, k]: values [rows, kpad], scales [kpad / 128, rows]."""
    values: object
    scales: object
    k: int


class Sparse24Fp8(NamedTuple):
    """2:4 operand [rows, k] (or a stack [experts, rows, k]): values [.., rows, kpad / 2],
    meta int32 [.., rows, kpad / 32], scales [.., ceil(rows / 128), kpad / 128]."""
    values: object
    meta: object
    scales: object
    k: int


def _pad(k: int) -> int:
    return -(-k // 128) * 128


def _blocks(k: int) -> int:
    return -(-k // 128)


def _placed(fn):
    """fn without its leading torch argument: run on its first argument's device, and on
    `stream` if one is given."""
    signature = inspect.signature(fn)
    params = list(signature.parameters.values())[1:]
    first = params[0].name

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        torch = _lib._torch()
        if not args and first not in kw:
            raise TypeError(f"{fn.__name__}() missing required argument: '{first}'")
        x = args[0] if args else kw[first]
        t = x[0] if isinstance(x, (tuple, list)) and x else x  # an operand's values, the first of a list
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{fn.__name__} needs CUDA (HIP) torch tensors")
        device = t.device
        if stream is None and device.index == torch.cuda.current_device():
            return fn(torch, *args, **kw)
        if stream is None:
            with torch.cuda.device(device):
                return fn(torch, *args, **kw)
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            return fn(torch, *args, **kw)

    call.__signature__ = signature.replace(
        parameters=params + [inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return call


def _run(torch, where, device, fn, *args):
    # the handle of the current stream; the public way builds a Stream object first (1.8 us,
    # a sixth of a small call)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    stream = raw(device.index) if raw else torch.cuda.current_stream(device).cuda_stream
    st = fn(*args, stream)
    if st != 0:
        raise TsenorError(st, where)


def _float_type(torch, t, name):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"{name} must be float32 or bfloat16")


def _matrix(torch, t, name, dim=2):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    if t.dim() != dim or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name} must be {dim}-D with unit column stride")


def _ld(t):
    """Leading dimension of a matrix (a single row may have any stride)."""
    return max(t.stride(-2), t.shape[-1]) if t.shape[-2] == 1 else t.stride(-2)


def _part(torch, t, dtype, shape, device, name, part=""):
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device
            or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{name}{part} must be a contiguous {dtype} tensor of shape {shape} on {device}")


def _dense(torch, a, device, name):
    """Checks a DenseFp8 operand; returns its number of rows."""
    if not isinstance(a, DenseFp8):
        raise TypeError(f"{name} must be a DenseFp8 operand (quant_fp8)")
    rows = a.values.shape[0]
    _part(torch, a.values, torch.float8_e4m3fn, (rows, _pad(a.k)), device, name, ".values")
    _part(torch, a.scales, torch.float8_e8m0fnu, (_blocks(a.k), rows), device, name, ".scales")
    return rows


def _sparse(torch, a, device, name, lead, rows=None):
    """Checks a Sparse24Fp8 operand with leading dimensions `lead`; returns its rows."""
    if not isinstance(a, Sparse24Fp8):
        raise TypeError(f"{name} must be a Sparse24Fp8 operand (compress24_fp8)")
    if rows is None:
        if a.values.dim() != len(lead) + 2:
            raise ValueError(f"{name}.values must have {len(lead) + 2} dimensions")
        rows = a.values.shape[-2]
    b = _blocks(a.k)
    _part(torch, a.values, torch.float8_e4m3fn, (*lead, rows, 64 * b), device, name, ".values")
    _part(torch, a.meta, torch.int32, (*lead, rows, 4 * b), device, name, ".meta")
    _part(torch, a.scales, torch.float8_e8m0fnu, (*lead, _blocks(rows), b), device, name, ".scales")
    return rows


def _span(t):
    """First byte, bytes of a row, bytes from row to row, bytes in all (a contiguous tensor of
    another dimension counts as one row)."""
    if t.dim() == 2:
        width, pitch = t.shape[1] * t.element_size(), _ld(t) * t.element_size()
        return t.data_ptr(), width, pitch, (t.shape[0] - 1) * pitch + width
    size = t.numel() * t.element_size()
    return t.data_ptr(), size, size, size


def _apart(out, x):
    """Refuses an `out` that shares bytes with the input x."""
    if out.numel() == 0 or x.numel() == 0:
        return
    (a, aw, ap, an), (b, bw, bp, bn) = _span(out), _span(x)
    if a + an <= b or b + bn <= a:
        return
    if ap == bp and aw <= (b - a) % ap <= ap - bw:  # columns of one buffer, side by side
        return
    if aw <= (b - a) % ap <= ap - bn or bw <= (a - b) % bp <= bp - an:  # one whole between two rows
        return
    raise ValueError("out overlaps an input")


def _end(t):
    """The address behind a matrix's last byte."""
    rows, cols = t.shape
    return t.data_ptr() + ((rows - 1) * t.stride(0) + cols) * t.element_size()


def _none_overlaps(out, inputs):
    """_apart for all of a call's inputs, the parts of operands among them.  Most lie before `out` or
    behind it: their addresses alone tell (_apart takes 3 us each, a small call 10)."""
    first, last = out.data_ptr(), _end(out)
    for x in inputs:
        if isinstance(x, tuple):
            for part in x[:-1]:  # contiguous
                p = part.data_ptr()
                if p < last and first < p + part.nbytes:
                    _apart(out, part)
        elif x is not None and x.data_ptr() < last and first < _end(x):
            _apart(out, x)


def _out(torch, out, shape, dtype, near, inputs):
    """A fresh result on the device of `near`, or `out` after checking it (and that it does not
    overlap any of the tensors `inputs`; an operand stands for its parts)."""
    if out is None:
        return near.new_empty(shape, dtype=dtype or torch.bfloat16)
    device = near.device
    _matrix(torch, out, "out")
    if tuple(out.shape) != shape or out.device != device or (dtype is not None and out.dtype != dtype):
        raise ValueError(f"out must be a tensor of shape {shape} on {device}"
                         + (f" and type {dtype}" if dtype is not None else ""))
    if shape[0] > 1 and out.stride(0) < shape[1]:
        raise ValueError("the rows of out overlap")
    _none_overlaps(out, inputs)
    return out


def _quant(torch, X, by_rows, by_cols):
    _matrix(torch, X, "X")
    dt = _float_type(torch, X, "X")
    rows, cols = X.shape
    if cols == 0:
        raise ValueError("X has no columns")
    new, e4m3, e8m0 = X.new_empty, torch.float8_e4m3fn, torch.float8_e8m0fnu
    rb, cb = -(-rows // 128), -(-cols // 128)
    a = b = av = as_ = bv = bs = None
    if by_rows:
        a = DenseFp8(new((rows, cb * 128), dtype=e4m3), new((cb, rows), dtype=e8m0), cols)
        av, as_ = a.values.data_ptr(), a.scales.data_ptr()
    if by_cols:
        b = DenseFp8(new((cols, rb * 128), dtype=e4m3), new((rb, cols), dtype=e8m0), rows)
        bv, bs = b.values.data_ptr(), b.scales.data_ptr()
    if rows:
        _run(torch, "tsenor_quant_fp8", X.device, lib().tsenor_quant_fp8, X.data_ptr(), dt, rows, cols,
             _ld(X), av, as_, bv, bs)
    return a, b


@_placed
def quant_fp8(torch, X, transpose: bool = False):
    """X (f32 or bf16 [rows, cols]) as a DenseFp8 operand with blocks along its
    rows; with transpose, X^T with blocks along X's columns (tsenor_quant_fp8)."""
    a, b = _quant(torch, X, not transpose, transpose)
    return b if transpose else a


@_placed
def quant_fp8_both(torch, X):
    """(quant_fp8(X), quant_fp8(X, transpose=True)) from one pass over X."""
    return _quant(torch, X, True, True)


def _compress(torch, W, mask, by_rows, by_cols):
    stacked = isinstance(W, torch.Tensor) and W.dim() == 3
    _matrix(torch, W, "W", 3 if stacked else 2)
    dt = _float_type(torch, W, "W")
    lead, (rows, cols) = tuple(W.shape[:-2]), W.shape[-2:]
    _part(torch, mask, torch.int32, (*lead, rows, (cols + 31) // 32), W.device, "mask")
    dev = W.device

    def new(r, k):
        b = _blocks(k)
        return Sparse24Fp8(W.new_empty((*lead, r, 64 * b), dtype=torch.float8_e4m3fn),
                           W.new_empty((*lead, r, 4 * b), dtype=torch.int32),
                           W.new_empty((*lead, _blocks(r), b), dtype=torch.float8_e8m0fnu), k)

    a = new(rows, cols) if by_rows else None
    t = new(cols, rows) if by_cols else None
    bad_a, bad_t = torch.zeros((2, 1), dtype=torch.int32, device=dev).unbind()
    if not stacked or W.shape[0]:
        _run(torch, "tsenor_compress24_fp8", dev, lib().tsenor_compress24_fp8, W.data_ptr(), dt,
             W.shape[0] if stacked else 1, W.stride(0) if stacked else 0, rows, cols, _ld(W),
             mask.data_ptr(), a and a.values.data_ptr(), a and a.meta.data_ptr(),
             a and a.scales.data_ptr(), t and t.values.data_ptr(), t and t.meta.data_ptr(),
             t and t.scales.data_ptr(), bad_a.data_ptr(), bad_t.data_ptr())
    return a, t, bad_a, bad_t


@_placed
def compress24_fp8(torch, W, mask, transpose: bool = False):
    """The 2:4 8-bit operand of W (or W^T) under its 2:4 mask (the int32 words of
    mask()); W f32 or bf16 [rows, cols] or a stack [experts, rows, cols] with a
    stack of masks.  Returns (Sparse24Fp8, bad), bad a CUDA int32 tensor with the
    number of groups that hold more than two kept entries."""
    a, t, bad_a, bad_t = _compress(torch, W, mask, not transpose, transpose)
    return (t, bad_t) if transpose else (a, bad_a)


@_placed
def compress24_fp8_both(torch, W, mask):
    """The operands of W and of W^T from one pass, with the same 8-bit numbers:
    (operand, operand_t, bad, bad_t)."""
    return _compress(torch, W, mask, True, True)


@_placed
def spmm24_fp8(torch, X, A, out=None, dtype=None):
    """Y = X A^T with A a Sparse24Fp8 operand [m, k] (tsenor_spmm24_fp8).  X: a
    DenseFp8 operand [n, k], or a bf16 or f32 tensor, which is quantised along
    its rows first.  Returns [n, m] in `dtype` (bf16 unless given or taken from
    `out`, which must not overlap X or A)."""
    ready = isinstance(X, DenseFp8)
    if ready:
        device = X.values.device
        n, k = _dense(torch, X, device, "X"), X.k
    else:
        _matrix(torch, X, "X")
        xt = _float_type(torch, X, "X")
        device, (n, k) = X.device, X.shape
    m = _sparse(torch, A, device, "A", ())
    if A.k != k:
        raise ValueError(f"X has {k} columns, A has {A.k}")
    out = _out(torch, out, (n, m), dtype, A.values, (X, A))
    yt = _float_type(torch, out, "out")
    if n == 0 or m == 0:
        return out
    if not ready and xt == BF16 and n <= 16:
        x, xtype, xs, ldx = X, BF16, None, _ld(X)
    else:
        q = X if ready else _quant(torch, X, True, False)[0]
        x, xtype, xs, ldx = q.values, E4M3, q.scales.data_ptr(), q.values.shape[1]
    _run(torch, "tsenor_spmm24_fp8", device, lib().tsenor_spmm24_fp8, x.data_ptr(), xtype, xs, n, ldx,
         A.values.data_ptr(), A.meta.data_ptr(), A.scales.data_ptr(), m, k, out.data_ptr(), yt, _ld(out))
    return out


@_placed
def gemm_fp8(torch, A, B, mask=None, out=None, dtype=None):
    """C = A B^T for DenseFp8 operands A [p, k] and B [q, k]; with a mask (int32
    words [p, ceil(q / 32)]) the removed entries are 0 (tsenor_gemm_fp8).  The
    masked weight gradient of Y = X W^T is
    gemm_fp8(quant_fp8(dY, transpose=True), quant_fp8(X, transpose=True), mask).
    Returns [p, q] in `dtype` (bf16 unless given or taken from `out`, which must
    not overlap A, B or the mask)."""
    if not isinstance(A, DenseFp8):
        raise TypeError("A must be a DenseFp8 operand (quant_fp8)")
    device = A.values.device
    p, q = _dense(torch, A, device, "A"), _dense(torch, B, device, "B")
    if A.k != B.k:
        raise ValueError(f"A has {A.k} columns, B has {B.k}")
    if mask is not None:
        _part(torch, mask, torch.int32, (p, (q + 31) // 32), device, "mask")
    out = _out(torch, out, (p, q), dtype, A.values, (A, B, mask))
    ct = _float_type(torch, out, "out")
    if p == 0 or q == 0:
        return out
    _run(torch, "tsenor_gemm_fp8", device, lib().tsenor_gemm_fp8, A.values.data_ptr(), A.scales.data_ptr(),
         p, B.values.data_ptr(), B.scales.data_ptr(), q, A.k,
         None if mask is None else mask.data_ptr(), out.data_ptr(), ct, _ld(out))
    return out


@_placed
def moe24_fp8(torch, x, router, gate, up, down, topk: int, out=None, return_routing: bool = False):
    """A mixture-of-experts layer for up to 64 tokens (tsenor_moe24_fp8): x bf16
    [n, d], router bf16 [experts, d], gate and up stacks of Sparse24Fp8 operands
    [experts, f, d], down [experts, d, f].  Returns y bf16 [n, d] (`out`, which
    must not overlap any of them), or with return_routing (y, ids int32 [n, topk],
    weights fp32 [n, topk])."""
    _matrix(torch, x, "x")
    _matrix(torch, router, "router")
    if x.dtype != torch.bfloat16 or router.dtype != torch.bfloat16:
        raise TypeError("x and router must be bfloat16")
    device, (n, d), experts = x.device, x.shape, router.shape[0]
    if router.device != device or router.shape[1] != d:
        raise ValueError(f"router must be [experts, {d}] on {device}")
    f = _sparse(torch, gate, device, "gate", (experts,))
    _sparse(torch, up, device, "up", (experts,), f)
    _sparse(torch, down, device, "down", (experts,), d)
    if gate.k != d or up.k != d or down.k != f:
        raise ValueError(f"gate and up must have {d} columns, down {f}")
    if not 1 <= topk <= experts:  # the library would see its low 32 bits
        raise TsenorError(4, "tsenor_moe24_fp8")  # TSENOR_ERR_PARAM
    out = _out(torch, out, (n, d), torch.bfloat16, x, (x, router, gate, up, down))
    ids = torch.empty((n, topk), dtype=torch.int32, device=device) if return_routing else None
    weights = torch.empty((n, topk), dtype=torch.float32, device=device) if return_routing else None
    size = lib().tsenor_moe24_fp8_workspace(n, d, f, experts, topk)
    work = torch.empty(size, dtype=torch.uint8, device=device)
    _run(torch, "tsenor_moe24_fp8", device, lib().tsenor_moe24_fp8, x.data_ptr(), n, _ld(x), d,
         router.data_ptr(), _ld(router), experts, topk, gate.values.data_ptr(), gate.meta.data_ptr(),
         gate.scales.data_ptr(), up.values.data_ptr(), up.meta.data_ptr(), up.scales.data_ptr(),
         down.values.data_ptr(), down.meta.data_ptr(), down.scales.data_ptr(), f, work.data_ptr(), size,
         out.data_ptr(), _ld(out), None if ids is None else ids.data_ptr(),
         None if weights is None else weights.data_ptr())
    return (out, ids, weights) if return_routing else out
