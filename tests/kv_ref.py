"""64-bit reference of the paged NVFP4 cache and its attention (numpy), written from the definitions in
include/bsg_kv.h: positions, pages, blocks and softmax one by one, no library code."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)])[:127]  # codes 0 .. 0x7E


def nearest(x, values):
    """Index of the nearest of the sorted values to each x >= 0, ties to the even index."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    down, up = x - values[lo], values[hi] - x
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def quantize(x, g=1.0):
    """Rows [..., n] -> (codes [..., n] with the sign in bit 3, scale codes [..., n/16])."""
    x = np.asarray(x, np.float64)
    y = (x * np.float64(np.float32(1.0) / np.float32(g))).astype(np.float32).astype(np.float64) if g != 1.0 else x
    b = y.reshape(*y.shape[:-1], -1, 16)
    amax = np.abs(b).max(-1)
    bad = np.isnan(amax)
    want = np.minimum(np.where(bad, 0.0, amax) / 6.0, 448.0)
    s = np.where(bad, 0x7F, nearest(want, E4M3))
    f = E4M3[np.minimum(s, 126)][..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        z = np.where((f > 0) & ~bad[..., None], np.abs(b) / f, 0.0)
    z = np.where(np.isnan(z), 0.0, np.minimum(z, 6.0))
    code = nearest(z, E2M1) | np.where(np.signbit(b), 8, 0)
    return code.reshape(y.shape).astype(np.uint8), s.astype(np.uint8)


def values(code, s, g=1.0):
    f = np.where(s == 0x7F, np.nan, E4M3[np.minimum(s, 126)])
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    return (v.reshape(*v.shape[:-1], -1, 16) * f[..., None]).reshape(v.shape) * np.float64(np.float32(g))


def rotate(x, pos, table, interleaved):
    """x [tokens][heads][D], pos [tokens], table [rows][2][R/2] -> rotated, each product and sum rounded to 32 bits."""
    x = np.asarray(x, np.float32).copy()
    if table is None:
        return x
    half = table.shape[2]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    cos, sin = table[pos, 0][:, None], table[pos, 1][:, None]
    x1, x2 = x[..., a].copy(), x[..., b].copy()
    with np.errstate(invalid="ignore", over="ignore"):
        x[..., a] = x1 * cos - x2 * sin
        x[..., b] = x2 * cos + x1 * sin
    return x


class Cache:
    """A cache's bytes with views of its parts."""

    def __init__(self, pages, heads, dim, page_tokens, fill=0, page_stride=0):
        self.dim, self.p, self.heads = dim, page_tokens, heads
        n = heads * page_tokens * dim * 9 // 8
        self.stride = page_stride or n
        self.bytes = np.full((pages, self.stride), fill, np.uint8)
        c = self.bytes[:, :n].reshape(pages, heads, -1)
        p, d = page_tokens, dim
        self.kc, self.vc = c[..., : p * d // 2].reshape(pages, heads, p, d // 2), None
        self.parts = [(0, (p, d // 2)), (p * d // 2, (p, d // 2)), (p * d, (p, d // 16)), (p * d + p * d // 16, (d // 16, p))]

    def part(self, page, head, which):
        """A writable view of one part (0 key codes, 1 value codes, 2 key scales, 3 value scales) of a page's head."""
        at, shape = self.parts[which]
        chunk = self.p * self.dim * 9 // 8
        return self.bytes[page, head * chunk + at: head * chunk + at + shape[0] * shape[1]].reshape(shape)

    def store(self, page, slot, head, is_v, code, s):
        packed = code[0::2] | (code[1::2] << 4)
        self.part(page, head, 1 if is_v else 0)[slot] = packed
        if is_v:
            self.part(page, head, 3)[:, slot] = s
        else:
            self.part(page, head, 2)[slot] = s

    def load(self, page, slot, head, is_v, g=1.0):
        packed = self.part(page, head, 1 if is_v else 0)[slot]
        code = np.empty(self.dim, np.uint8)
        code[0::2], code[1::2] = packed & 15, packed >> 4
        s = self.part(page, head, 3)[:, slot] if is_v else self.part(page, head, 2)[slot]
        return values(code, s, g)


def positions(q_start, kv_len):
    """(sequence, position) of every new token."""
    out = []
    for b in range(len(kv_len)):
        n = q_start[b + 1] - q_start[b]
        out += [(b, kv_len[b] - n + i) for i in range(n)]
    return out


def attend(q, cache, q_start, kv_len, pages, kv_heads, scale=None, causal=True, window=0, softcap=0.0, k_scale=1.0, v_scale=1.0):
    """q [tokens][q_heads][D] float64 -> (out, lse) float64."""
    tokens, hq, d = q.shape
    g = hq // kv_heads
    scale = d ** -0.5 if scale is None else scale
    out, lse = np.zeros(q.shape), np.full((tokens, hq), -np.inf)
    held = {}
    for t, (b, pos) in enumerate(positions(q_start, kv_len)):
        last = pos if causal else kv_len[b] - 1
        first = max(0, pos - window + 1) if window else 0
        if last < first:
            continue
        for h in range(kv_heads):
            if (b, h) not in held:
                at = [(pages[b][p // cache.p], p % cache.p) for p in range(kv_len[b])]
                held[b, h] = (np.array([cache.load(pg, sl, h, False, k_scale) for pg, sl in at]),
                              np.array([cache.load(pg, sl, h, True, v_scale) for pg, sl in at]))
            k, v = (x[first:last + 1] for x in held[b, h])
            for j in range(h * g, (h + 1) * g):
                with np.errstate(invalid="ignore"):
                    s = (k @ q[t, j]) * scale
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                    m = s.max()
                    e = np.exp(s - (0.0 if m == -np.inf else m))
                    total = e.sum()
                    out[t, j] = (e @ v) / total if total != 0 else 0.0
                    lse[t, j] = m + np.log(total) if total != 0 else -np.inf
    return out, lse
