"""64-bit reference of the expert layer (numpy), from the formulas in include/bsg_moe.h."""
from __future__ import annotations

import numpy as np

from oracle.oracle import dequant_mxfp8, dequant_nvfp4


def moe(fmt, x, router, w13, s13, w2, s2, top_k, a13=None, a2=None, renormalize=True):
    """x, router float64; codes and scales uint8 per expert -> (out, ids, weights)."""
    T, H = x.shape
    E = router.shape[0]
    inter = w2.shape[-1] * (2 if fmt == "nvfp4" else 1)

    def rows(codes, scales):
        return dequant_nvfp4(codes, scales, codes.shape[1] * 2) if fmt == "nvfp4" else dequant_mxfp8(codes, scales)

    out, ids, weights = np.zeros((T, H)), np.zeros((T, top_k), np.int32), np.zeros((T, top_k))
    held = {}
    for t in range(T):
        logits = router @ x[t]
        p = np.exp(logits - logits.max())
        p /= p.sum()
        ids[t] = np.argsort(-logits, kind="stable")[:top_k]
        weights[t] = p[ids[t]] / (p[ids[t]].sum() if renormalize else 1.0)
        for j, e in enumerate(ids[t]):
            if e not in held:
                held[e] = (rows(w13[e], s13[e]) * (1.0 if a13 is None else float(a13[e])), rows(w2[e], s2[e]) * (1.0 if a2 is None else float(a2[e])))
            m13, m2 = held[e]
            gu = m13 @ x[t]
            gate, up = gu[:inter], gu[inter:]
            with np.errstate(over="ignore"):
                out[t] += weights[t, j] * (m2 @ (gate / (1.0 + np.exp(-gate)) * up))
    return out, ids, weights
