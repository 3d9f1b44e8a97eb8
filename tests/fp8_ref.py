"""The 8-bit formats and products in numpy and 64 bits, from their definition
(include/tsenor_fp8.h); shares no code with the library.  Imported by tests only."""
import numpy as np


def _decode_table():
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = np.nan if (b & 0x7F) == 0x7F else (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        v[b] = -x if b & 0x80 else x
    return v


E4M3 = _decode_table()
_POS = E4M3[:0x7F]                       # 0 .. 448 ascending
_MID = (_POS[1:] + _POS[:-1]) / 2


def round_e4m3(x):
    """Codes of the nearest e4m3 numbers, ties to the even code; non-finite -> NaN."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    lo = np.searchsorted(_MID, a, side="left")        # ties stay at the lower code
    tie = (lo < len(_MID)) & (a == _MID[np.minimum(lo, len(_MID) - 1)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def exponent(amax):
    """Least s >= -127 with amax <= 448 * 2^s, 0 for 0; by comparison only."""
    amax = np.asarray(amax, np.float64)
    s = np.full(amax.shape, -127)
    for k in range(-127, 122):
        s = np.where(amax > 448.0 * 2.0 ** k, k + 1, s)
    return np.where(amax == 0, 0, s)


def pad(k):
    return -(-k // 128) * 128


def finite_abs(x):
    return np.where(np.isfinite(x), np.abs(np.where(np.isfinite(x), x, 0.0)), 0.0)


def quant(x):
    """(codes [r, kpad], scale bytes [kpad/128, r], dequantised fp64 [r, kpad])."""
    r, c = x.shape
    full = np.zeros((r, pad(c)))
    full[:, :c] = x
    s = exponent(finite_abs(full).reshape(r, -1, 128).max(-1))
    wide = np.repeat(2.0 ** s, 128, axis=1)
    codes = round_e4m3(full / wide)
    return codes, (s + 127).astype(np.uint8).T, E4M3[codes] * wide


def compress(w, keep):
    """(codes [r, kpad/2], meta [r, kpad/32], scale bytes, groups with > 2, dense fp64 [r, kpad])."""
    r, c = w.shape
    R, C = pad(r), pad(c)
    full, k = np.zeros((R, C)), np.zeros((R, C), bool)
    full[:r, :c], k[:r, :c] = np.where(keep, w, 0.0), keep
    s = exponent(finite_abs(full).reshape(R // 128, 128, C // 128, 128).max((1, 3)))
    wide = np.repeat(np.repeat(2.0 ** s, 128, 0), 128, 1)
    q = round_e4m3(full / wide)
    codes = np.zeros((r, C // 2), np.uint8)
    meta = np.zeros((r, C // 32), np.uint32)
    dense = np.zeros((r, C))
    bad = 0
    for i in range(r):
        for g in range(C // 4):
            pos = [j for j in range(4) if k[i, 4 * g + j]]
            bad += len(pos) > 2
            pos = pos[:2]
            for slot, j in enumerate(pos):
                codes[i, 2 * g + slot] = q[i, 4 * g + j]
                dense[i, 4 * g + j] = E4M3[q[i, 4 * g + j]] * wide[i, 4 * g + j]
            p = (pos + [3, 2] if len(pos) == 1 and pos[0] != 3 else pos + [2]) if len(pos) == 1 else \
                (pos if pos else [0, 1])
            meta[i, g // 8] |= np.uint32((p[0] | (p[1] << 2)) << (4 * (g % 8)))
    return codes, meta, (s + 127).astype(np.uint8), bad, dense


def expand(codes, meta, scales, k=None):
    """Dense fp64 [r, kpad] of a 2:4 operand's arrays."""
    r, half = codes.shape
    dense = np.zeros((r, 2 * half))
    for slot in range(half):
        p = (meta[:, slot // 16] >> np.uint32(2 * (slot % 16))) & 3
        dense[np.arange(r), 4 * (slot // 2) + p] += E4M3[codes[:, slot]]
    s = 2.0 ** (scales.astype(np.float64) - 127)
    s = np.repeat(np.repeat(s, 128, 0)[:r], 128, 1)
    return dense * s


def pack_mask(keep):
    r, c = keep.shape
    w = np.zeros((r, (c + 31) // 32), np.uint32)
    for j in range(c):
        w[:, j // 32] |= keep[:, j].astype(np.uint32) << np.uint32(j % 32)
    return w


def random24(rng, rows, cols):
    """A 2:4 mask with two ones in every row and column of each 4 x 4 block."""
    keep = np.zeros((rows, cols), bool)
    base = np.array([[1, 1, 0, 0], [1, 1, 0, 0], [0, 0, 1, 1], [0, 0, 1, 1]], bool)
    for i in range(0, rows, 4):
        for j in range(0, cols, 4):
            keep[i:i + 4, j:j + 4] = base[rng.permutation(4)][:, rng.permutation(4)]
    return keep
