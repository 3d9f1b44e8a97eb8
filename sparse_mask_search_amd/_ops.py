"""Binding of the dense operators of masked models (include/tsenor_ops.h):
products grouped by expert, 8-bit integer products, clipping of gradients.

Rows of a grouped operand are sorted by expert; ``ends`` (int32 [experts], on the
device) holds the row behind each expert's last one.  With ``stream`` a call runs
on that stream and takes its memory there; otherwise it runs on the current
stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import _lib
from ._fp8 import _apart, _blocks, _float_type, _ld, _matrix, _pad, _part, _placed, _run
from ._lib import BF16, F32, lib

INT8 = 3


def _in_one_launch(rows, k, m):
    """Whether bf16 tokens become integers inside the product: every workgroup of 16 columns does it for itself, which
    costs 0.8 us a further token up to 4096 columns (a workgroup for each CU), 1.9 at 11008 and 4.2 at 32000;
    a launch of its own costs 3 us, and 5 of the host's.  Measured (us), inside / before: called one by one 1 token
    4096 x 4096 9.5 / 14.3, 4 tokens 10.2 / 14.0, 8 tokens 14.4 / 14.0, 12 tokens 512 x 512 12.7 / 14.1, 16 tokens 4096 x 2048
    18.7 / 14.0, 3 tokens 11008 x 4096 16.1 / 16.0, 1 token 32000 x 4096 27.7 / 30.4, 2 tokens 32.7 / 30.5; in a graph, the
    same, 7.7 / 10.3, 10.3 / 10.9, 14.6 / 11.1, 12.2 / 6.2, 18.8 / 9.9, 16.6 / 16.8, 29.0 / 31.2, 33.3 / 31.4.  Past four
    tokens a graph wants the launch and calls one by one do not: eight lie between."""
    return (rows == 1 or rows <= 8 and rows * m <= 32768) and rows * _pad(k) <= 32768


class DenseInt8(NamedTuple):
    """8-bit integer operand [rows, k] (or a stack [experts, rows, k]): values int8
    [.., rows, kpad], scales fp32 [.., rows]; a row stands for values * scale."""
    values: object
    scales: object
    k: int


def _ends(torch, ends, device, experts=None):
    if (not isinstance(ends, torch.Tensor) or ends.dtype != torch.int32 or ends.device != device or ends.dim() != 1
            or not ends.is_contiguous() or (experts is not None and ends.shape[0] != experts)):
        raise ValueError(f"ends must be a contiguous int32 tensor of shape "
                         f"{'[experts]' if experts is None else (experts,)} on {device}")
    return ends.shape[0]


def _bf16_matrix(torch, t, name, device=None, dim=2):
    _matrix(torch, t, name, dim)
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _stack_strides(t):
    """From matrix to matrix of a stack, from row to row (a single one may have any stride)."""
    ld = t.shape[-1] if t.shape[-2] == 1 else t.stride(-2)
    return (t.shape[-2] * ld if t.shape[0] == 1 else t.stride(0)), ld


def _last(t):
    """The address behind a tensor's last byte."""
    return t.data_ptr() + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _separate(out, inputs):
    """Refuses an `out` that shares bytes with an input (None: not given)."""
    if out.numel() == 0:
        return
    first, last = out.data_ptr(), _last(out)
    for x in inputs:
        if x is None or x.numel() == 0:
            continue
        if x.data_ptr() < last and first < _last(x):
            if out.dim() == 2 and (x.dim() == 2 or x.is_contiguous()):
                _apart(out, x)  # matrices may lie side by side in one buffer
            else:
                raise ValueError("out overlaps an input")


def _result(torch, out, shape, dtype, near, inputs):
    """A fresh result on the device of `near`, or `out` after its checks."""
    if out is None:
        return near.new_empty(shape, dtype=dtype or torch.bfloat16)
    _matrix(torch, out, "out", len(shape))
    if tuple(out.shape) != shape or out.device != near.device or (dtype is not None and out.dtype != dtype):
        raise ValueError(f"out must be a tensor of shape {shape} on {near.device}"
                         + (f" and type {dtype}" if dtype is not None else ""))
    if shape[-2] > 1 and out.stride(-2) < shape[-1]:
        raise ValueError("the rows of out overlap")
    if len(shape) == 3 and shape[0] > 1 and out.stride(0) < shape[1] * _stack_strides(out)[1]:
        raise ValueError("the matrices of out overlap")
    _separate(out, inputs)
    return out


@_placed
def grouped_mm(torch, X, W, ends, transpose: bool = False, out=None, dtype=None):
    """Products grouped by expert (tsenor_grouped_mm): Y[r] = X[r] W[e]^T for the expert e
    that owns row r, W bf16 [experts, m, k]; with transpose, Y[r] = X[r] W[e], W
    [experts, k, m] (the data gradient of the former).  X bf16 [rows, k], rows sorted by
    expert; rows behind ends[-1] come out as zeros.  Returns [rows, m] in `dtype` (bf16
    unless given or taken from `out`, which must not overlap X, W or ends)."""
    _bf16_matrix(torch, X, "X")
    device, (rows, k) = X.device, X.shape
    _bf16_matrix(torch, W, "W", device, 3)
    experts, m, wk = W.shape
    if transpose:
        m, wk = wk, m
    if wk != k:
        raise ValueError(f"X has {k} columns, W needs {wk}")
    _ends(torch, ends, device, experts)
    out = _result(torch, out, (rows, m), dtype, X, (X, W, ends))
    yt = _float_type(torch, out, "out")
    if rows == 0 or m == 0:
        return out
    if k == 0 or experts == 0:
        raise ValueError("X has no columns" if k == 0 else "W holds no expert")
    stride, ldw = _stack_strides(W)
    _run(torch, "tsenor_grouped_mm", device, lib().tsenor_grouped_mm, X.data_ptr(), rows, _ld(X), W.data_ptr(),
         1 if transpose else 0, experts, stride, ldw, m, k, ends.data_ptr(), out.data_ptr(), yt, _ld(out))
    return out


@_placed
def grouped_wgrad(torch, dY, X, ends, mask=None, out=None, dtype=None):
    """Weight gradients of grouped_mm(X, W, ends): dW[e] = dY_e^T X_e over the rows of expert e
    (tsenor_grouped_wgrad), dY bf16 [rows, m], X bf16 [rows, k]; with a mask (int32 words
    [experts, m, ceil(k / 32)], those of mask() expert by expert) the removed entries are 0.  Returns
    [experts, m, k] in `dtype` (bf16 unless given or taken from `out`, which must not
    overlap any of them); an expert without rows has zeros."""
    _bf16_matrix(torch, dY, "dY")
    device, (rows, m) = dY.device, dY.shape
    _bf16_matrix(torch, X, "X", device)
    if X.shape[0] != rows:
        raise ValueError(f"dY has {rows} rows, X has {X.shape[0]}")
    k, experts = X.shape[1], _ends(torch, ends, device)
    if mask is not None:
        _part(torch, mask, torch.int32, (experts, m, (k + 31) // 32), device, "mask")
    out = _result(torch, out, (experts, m, k), dtype, X, (dY, X, ends, mask))
    ct = _float_type(torch, out, "out")
    if out.numel() == 0:
        return out
    stride, ldc = _stack_strides(out)
    _run(torch, "tsenor_grouped_wgrad", device, lib().tsenor_grouped_wgrad, dY.data_ptr(), _ld(dY), X.data_ptr(),
         _ld(X), rows, experts, m, k, ends.data_ptr(), None if mask is None else mask.data_ptr(), out.data_ptr(),
         ct, stride, ldc)
    return out


def _quantised(torch, X):
    stacked = isinstance(X, torch.Tensor) and X.dim() == 3
    _matrix(torch, X, "X", 3 if stacked else 2)
    dt = _float_type(torch, X, "X")
    lead, (rows, k) = tuple(X.shape[:-2]), X.shape[-2:]
    if k == 0:
        raise ValueError("X has no columns")
    a = DenseInt8(X.new_empty((*lead, rows, _pad(k)), dtype=torch.int8),
                  X.new_empty((*lead, rows), dtype=torch.float32), k)
    if X.numel():
        stride, ld = _stack_strides(X) if stacked else (0, _ld(X))
        _run(torch, "tsenor_quant_int8", X.device, lib().tsenor_quant_int8, X.data_ptr(), dt,
             X.shape[0] if stacked else 1, stride, rows, k, ld, a.values.data_ptr(), a.scales.data_ptr())
    return a


@_placed
def quant_int8(torch, X):
    """X (f32 or bf16 [rows, k], or a stack [experts, rows, k]) as a DenseInt8 operand: each
    row to integers of its largest magnitude / 127 (tsenor_quant_int8)."""
    return _quantised(torch, X)


def _integers(torch, a, device, name, lead):
    """Checks a DenseInt8 operand with leading dimensions `lead`; returns its rows."""
    if not isinstance(a, DenseInt8):
        raise TypeError(f"{name} must be a DenseInt8 operand (quant_int8)")
    if a.values.dim() != len(lead) + 2:
        raise ValueError(f"{name}.values must have {len(lead) + 2} dimensions")
    rows = a.values.shape[-2]
    _part(torch, a.values, torch.int8, (*lead, rows, 128 * _blocks(a.k)), device, name, ".values")
    _part(torch, a.scales, torch.float32, (*lead, rows), device, name, ".scales")
    return rows


@_placed
def gemm_int8(torch, X, A, ends=None, out=None, dtype=None):
    """Y = X A^T in 8-bit integers with a scale for each row of X and of A
    (tsenor_gemm_int8).  A: a DenseInt8 operand [m, k], or with `ends` a stack [experts, m, k]
    whose expert e multiplies the rows that it owns (rows behind ends[-1] come out as
    zeros).  X: a DenseInt8 operand [rows, k], or a bf16 or f32 tensor, which is quantised
    first.  Returns [rows, m] in `dtype` (bf16 unless given or taken from `out`, which must
    not overlap X, A or ends)."""
    ready = isinstance(X, DenseInt8)
    if ready:
        device = X.values.device
        rows, k = _integers(torch, X, device, "X", ()), X.k
    else:
        _matrix(torch, X, "X")
        xt = _float_type(torch, X, "X")
        device, (rows, k) = X.device, X.shape
    experts = 1 if ends is None else _ends(torch, ends, device)
    m = _integers(torch, A, device, "A", () if ends is None else (experts,))
    if A.k != k:
        raise ValueError(f"X has {k} columns, A has {A.k}")
    if out is None:
        out = A.values.new_empty((rows, m), dtype=dtype or torch.bfloat16)
    else:
        out = _result(torch, out, (rows, m), dtype, A.values,
                      (*(X[:2] if ready else (X,)), A.values, A.scales, ends))
    yt = _float_type(torch, out, "out")
    if rows == 0 or m == 0:
        return out
    if k == 0 or experts == 0:
        raise ValueError("X has no columns" if k == 0 else "A holds no expert")
    if ready:
        x, xtype, xs, ldx = X.values.data_ptr(), INT8, X.scales.data_ptr(), X.values.shape[1]
    elif xt == BF16 and ends is None and _in_one_launch(rows, k, m):
        x, xtype, xs, ldx = X.data_ptr(), BF16, None, _ld(X)
    else:  # quantised into one buffer, scales behind the values
        ldx = _pad(k)
        q = torch.empty(rows * (ldx + 4), dtype=torch.int8, device=device)
        x, xtype, xs = q.data_ptr(), INT8, q.data_ptr() + rows * ldx
        _run(torch, "tsenor_quant_int8", device, lib().tsenor_quant_int8, X.data_ptr(), xt, 1, 0, rows, k, _ld(X), x, xs)
    _run(torch, "tsenor_gemm_int8", device, lib().tsenor_gemm_int8, x, xtype, xs, rows, ldx,
         A.values.data_ptr(), A.scales.data_ptr(), experts, m, k, None if ends is None else ends.data_ptr(),
         out.data_ptr(), yt, _ld(out))
    return out


def _as_rows(t, name):
    """A gradient as rows along its last dimension: (rows, columns, leading dimension)."""
    if t.is_contiguous():
        cols = t.shape[-1] if t.dim() else 1
        return (t.numel() // cols if cols else 0), cols, cols
    if t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] == 1) and t.stride(0) >= t.shape[1]:
        return t.shape[0], t.shape[1], t.stride(0)
    raise ValueError(f"{name} must be contiguous, or a matrix with unit column stride")


def _as_any(t, name):
    """A gradient without a mask: its entries in any order."""
    if t.dim() == 2 and t.stride(1) != 1 and t.stride(0) == 1 and t.stride(1) >= t.shape[0]:
        return t.shape[1], t.shape[0], t.stride(1)  # column by column
    return _as_rows(t, name)


def _matrix_of(t):
    """A gradient as the matrix that _apart looks at."""
    return t.t() if t.dim() == 2 and t.stride(1) != 1 and t.stride(0) == 1 else t


def _no_two(spans):
    """Refuses spans (first byte, byte behind the last, written, tensor) of which one that is written
    shares bytes with another."""
    spans.sort(key=lambda s: s[:2])
    end = 0
    for s in spans:
        if s[0] < end:
            break
        end = s[1]
    else:
        return  # all apart
    open_, end = [], 0
    for s in spans:
        if s[0] >= end:
            open_ = []
        for o in open_:
            if (s[2] or o[2]) and s[0] < o[1]:
                try:
                    _apart(_matrix_of(s[3]), _matrix_of(o[3]))
                except ValueError:
                    raise ValueError("a gradient that is written overlaps another tensor of the call") from None
        open_.append(s)
        end = max(end, s[1])


def _grad_list(torch, grads, masks, out, write):
    """The C descriptors of a list of gradients, eight 64-bit words each; if they are written, no two may
    overlap.  (A call on a small model's gradients is bound by this loop, 2 us a tensor.)"""
    if not isinstance(grads, (list, tuple)):
        raise TypeError("grads must be a list of tensors")
    n = len(grads)
    if masks is not None and len(masks) != n:
        raise ValueError("masks must hold one entry (a mask or None) per gradient")
    if out is not None and len(out) != n:
        raise ValueError("out must hold one tensor per gradient")
    device, words, spans = grads[0].device, [], []
    Tensor, f32, bf16, i32 = torch.Tensor, torch.float32, torch.bfloat16, torch.int32
    for i, g in enumerate(grads):
        if not isinstance(g, Tensor) or g.device != device:
            raise TypeError(f"grads[{i}] must be a tensor on {device}")
        dtype, shape = g.dtype, g.shape
        if dtype is not f32 and dtype is not bf16:
            raise TypeError(f"grads[{i}] must be float32 or bfloat16")
        o = g if out is None else out[i]
        if o is not g and (not isinstance(o, Tensor) or o.dtype is not dtype or o.shape != shape or o.device != device):
            raise ValueError(f"out[{i}] must be a tensor like grads[{i}]")
        m = None if masks is None else masks[i]
        if m is not None:
            want = (*shape[:-1], (shape[-1] + 31) // 32) if shape else None
            if (not isinstance(m, Tensor) or m.dtype is not i32 or m.shape != want or m.device != device
                    or not m.is_contiguous()):
                raise ValueError(f"masks[{i}] must be a contiguous int32 tensor of shape {want} on {device}")
        ptr, flat = g.data_ptr(), g.is_contiguous()
        to = ptr if o is g else o.data_ptr()
        if flat and (o is g or o.is_contiguous()):
            size = g.nbytes
            if m is None:
                rows, cols = 1, g.numel()
            else:
                cols = shape[-1]
                rows = g.numel() // cols if cols else 0
            ld = ldo = cols
            last, olast = ptr + size, to + size
        else:
            if m is None and (o is g or o.stride() == g.stride()):
                rows, cols, ld = _as_any(g, f"grads[{i}]")
                ldo = ld
            else:
                rows, cols, ld = _as_rows(g, f"grads[{i}]")
                ldo = ld if o is g else _as_rows(o, f"out[{i}]")[2]
            last, olast = _last(g), _last(o)
        words += (ptr, to, 0 if m is None else m.data_ptr(), F32 if dtype is f32 else BF16, rows, cols, ld, ldo)
        if write and rows and cols:
            spans.append((to, olast, True, o))
            if to != ptr:
                spans.append((ptr, last, False, g))
            if m is not None:
                spans.append((words[-6], words[-6] + m.nbytes, False, m))
    if write:
        _no_two(spans)
    return device, words


def _clip(torch, grads, masks, out, max_norm):
    write = max_norm is not None
    device, words = _grad_list(torch, grads, masks, out, write)
    n = len(grads)
    table = (ctypes.c_int64 * len(words))(*words)
    size = lib().tsenor_grads_workspace(n)
    work = torch.empty(size // 4 + 1, dtype=torch.float32, device=device)  # the norm lies behind the partial sums
    start = work.data_ptr()
    if write:
        _run(torch, "tsenor_clip_grads", device, lib().tsenor_clip_grads, table, n, float(max_norm), start, size,
             start + size)
    else:
        _run(torch, "tsenor_grad_norm", device, lib().tsenor_grad_norm, table, n, start, size, start + size)
    return work[size // 4]


@_placed
def grad_norm(torch, grads, masks=None):
    """The norm of a list of gradients (f32 or bf16 tensors of any shape) in 64 bits, as an fp32
    scalar on their device (tsenor_grad_norm).  masks: one entry per gradient, None or
    the int32 words [.., rows, ceil(cols / 32)] of its mask; removed entries do not count."""
    return _clip(torch, grads, masks, None, None)


@_placed
def clip_grads(torch, grads, max_norm, masks=None, out=None):
    """Scales a list of gradients by max_norm / norm where grad_norm(grads, masks) passes
    max_norm, and clears what the masks remove (tsenor_clip_grads): in place, or into
    the tensors `out`.  No tensor that is written may overlap another one of the call.  Returns the norm
    from before, as an fp32 scalar on their device; nothing waits for it."""
    return _clip(torch, grads, masks, out, max_norm)
