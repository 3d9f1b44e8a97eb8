"""The operators of include/tsenor_ops.h in numpy and 64 bits, from their definition; shares
no code with the library.  Imported by tests only."""
import numpy as np


def bounds(ends, rows):
    """(first, end) of every expert, entries of `ends` as they count."""
    e = np.maximum.accumulate(np.clip(np.asarray(ends, np.int64), 0, rows))
    return list(zip([0] + e[:-1].tolist(), e.tolist()))


def grouped_mm(x, w, ends, transpose):
    """Y, and the sums of magnitudes that bound its rounding."""
    m = w.shape[2] if transpose else w.shape[1]
    y, s = np.zeros((x.shape[0], m)), np.zeros((x.shape[0], m))
    for e, (a, b) in enumerate(bounds(ends, x.shape[0])):
        we = w[e] if transpose else w[e].T
        y[a:b], s[a:b] = x[a:b] @ we, np.abs(x[a:b]) @ np.abs(we)
    return y, s


def grouped_wgrad(dy, x, ends, keep=None):
    parts = bounds(ends, x.shape[0])
    dw = np.stack([dy[a:b].T @ x[a:b] for a, b in parts])
    s = np.stack([np.abs(dy[a:b]).T @ np.abs(x[a:b]) for a, b in parts])
    return (dw, s) if keep is None else (np.where(keep, dw, 0.0), np.where(keep, s, 0.0))


def pad(k):
    return -(-k // 128) * 128


def quant_int8(x):
    """(int8 [.., kpad], scales fp32) of float32 values.  x * 127 is exact in 64 bits, and the quotient's
    rounding (2^-53) is far below its distance from a half that it is not (2^-32)."""
    x64 = x.astype(np.float64)
    good = np.isfinite(x).all(-1)
    amax = np.where(good, np.abs(np.where(np.isfinite(x64), x64, 0.0)).max(-1), 0.0)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where((good & (amax > 0))[..., None], np.rint(x64 * 127.0 / amax[..., None]), 0.0)
    out = np.zeros((*x.shape[:-1], pad(x.shape[-1])), np.int8)
    out[..., :x.shape[-1]] = np.nan_to_num(q)
    scale = amax.astype(np.float32) / np.float32(127.0)
    return out, np.where(good, scale, np.float32(np.nan)).astype(np.float32)


def gemm_int8(x, xs, a, as_):
    """fp32 results, bit for bit before the output's rounding."""
    sums = x.astype(np.int64) @ a.astype(np.int64).T
    with np.errstate(invalid="ignore", over="ignore"):
        return sums.astype(np.float32) * xs[:, None] * as_[None, :]


def pack_mask(keep):
    *lead, c = keep.shape
    w = np.zeros((*lead, (c + 31) // 32), np.uint32)
    for j in range(c):
        w[..., j // 32] |= keep[..., j].astype(np.uint32) << np.uint32(j % 32)
    return w
