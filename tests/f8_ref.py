"""64-bit reference of the E4M3 products with a scale for each block of 128 (numpy), written from the definitions in
include/bsg_f8.h, no library code; and bounds of what the kernels may be off by."""
from __future__ import annotations

import numpy as np

from kv_ref import E4M3, nearest

BLOCK = 128
U32 = 2.0 ** -24
# Half a step of the output, relative to the value, and of its subnormal numbers.
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}
FEW = 16   # tokens up to which products are of widened codes (exact, with sums in fp32)
WIDE = 64  # ... and those whose results become codes


def blocks(n):
    return -(-n // BLOCK)


def values(codes):
    """Doubles of E4M3 codes."""
    codes = np.asarray(codes, np.uint8)
    v = np.where((codes & 127) == 127, np.nan, E4M3[np.minimum(codes & 127, 126)])
    return np.where(codes & 128, -v, v)


def quantize(x):
    """Rows [T][C] -> codes uint8 [T][C], scales [B][T]: the least power of two s >= 2^-126 with max|x| <= 448 s."""
    x = np.asarray(x, np.float64)
    codes, scales = np.zeros(x.shape, np.uint8), np.zeros((blocks(x.shape[1]), x.shape[0]))
    for b in range(len(scales)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        most = np.abs(part).max(1)
        fine = np.isfinite(most)
        frac, e = np.frexp(np.where(fine, most, 0.0))  # most = frac 2^e, 1/2 <= frac < 1; 448 = 7/8 2^9
        s = np.where(frac > 0, np.maximum(e - 9 + (frac > 0.875), -126), -126)
        scales[b] = np.ldexp(1.0, s)
        with np.errstate(invalid="ignore"):
            z = np.where(fine[:, None], np.abs(part) / scales[b][:, None], 0.0)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = np.where(fine[:, None], nearest(z, E4M3) | np.where(np.signbit(part), 128, 0), 0x7F)
    return codes, scales


def row_values(codes, scales):
    """Doubles of rows [T][C] with scales [B][T or more]."""
    return values(codes) * np.repeat(scales[:, :len(codes)].T, BLOCK, 1)[:, :codes.shape[1]]


def weight_values(codes, scales):
    """Doubles of weights [N][K] with scales [B(N)][B(K)]."""
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), BLOCK, 0)[:codes.shape[0]], BLOCK, 1)[:, :codes.shape[1]]
    return values(codes) * s


def sum_bound(k, few, exact_range=False):
    """How far a sum of k scaled products may be off, in units of the sum of their magnitudes: a rounding to fp32 for each
    product at the most and three for the scales; where the codes are not widened (few) the matrix instruction also aligns
    every 8 products to the largest and drops what lies 2^-13 below, 2^-10 of it for all 8, unless they span few bits
    (exact_range)."""
    return (k + 4) * U32 + (0.0 if few or exact_range else 2.0 ** -10)


def product(x, w, bias=None):
    """(x w^T + bias, the sum of the magnitudes) of doubles."""
    y, s = x @ w.T, np.abs(x) @ np.abs(w).T
    return (y, s) if bias is None else (y + bias, s + np.abs(bias))


def silu(x):
    return x / (1.0 + np.exp(-x))


def _changes(h, d):
    """How far the quantised value of each h may be from quantize(h)'s where h is off by up to d: every magnitude of a block
    moves by its own d, so the scale is the least or the greatest power of two that any of them allows."""
    codes, scales = quantize(h)
    held = row_values(codes, scales)
    out = np.zeros(h.shape)
    for b in range(len(scales)):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        most = np.abs(h[:, at]) + d[:, at]
        least = np.maximum(np.abs(h[:, at]) - d[:, at], 0.0)
        for end in (most, least):
            s = quantize(np.concatenate([end, np.zeros((len(h), BLOCK - end.shape[1]))], 1))[1][0][:, None]
            for v in (h[:, at] - d[:, at], h[:, at], h[:, at] + d[:, at]):
                q = np.where(v < 0, -1, 1) * E4M3[nearest(np.minimum(np.abs(v) / s, 448.0), E4M3)] * s
                out[:, at] = np.maximum(out[:, at], np.abs(q - held[:, at]))
    return out


def ffn(x, w1, w3, w2, exact_range=False):
    """(the block's output, how far the kernels' may be off before it is rounded) for doubles x, w1, w3 [I][H], w2 [H][I]."""
    few = len(x) <= WIDE
    xv = row_values(*quantize(x))
    (gate, sg), (up, su) = product(xv, w1), product(xv, w3)
    c = sum_bound(x.shape[1], few, exact_range)
    dg, du = c * sg, c * su
    h = silu(gate) * up
    # |SiLU'| < 1.1; SiLU's exponential, sum and reciprocal cost 8 roundings and the exponent's own, |gate| of them; two more
    # for the products
    d = 1.1 * dg * (np.abs(up) + du) + np.abs(silu(gate)) * du + np.abs(h) * (10 + np.abs(gate)) * U32 + 1e-38
    hv = row_values(*quantize(h))
    y, s = product(hv, w2)
    off = _changes(h, d)
    return y, sum_bound(h.shape[1], len(x) <= FEW) * (s + off @ np.abs(w2).T) + off @ np.abs(w2).T
