"""Plain reference of the verify step from probabilities and given random
numbers [P2 39.4, Listing 39.4; P3 "The Algorithm"], in float64, one sequence
at a time. Statuses as include/tsr.h (verify_probs) lists them."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

OK, NONFINITE, EMPTY, BADTOKEN, BADPARAM = range(5)


@dataclass
class Result:
    tokens: np.ndarray
    accepted: int
    status: int
    margin: float     # how near the draw came to the neighbouring token, relative to the sum


def _is_probability(x):
    return np.isfinite(x) & (x >= 0)


def verify_probs_row(p, q, drafts, n_drafts, accept_u, draw_u) -> Result:
    """p [K+1, V], q [K, V] or None, drafts [K], accept_u [K]."""
    K = len(drafts)
    p = np.asarray(p, dtype=np.float64)
    V = p.shape[1]

    def bad(status):
        return Result(np.full(K + 1, -1, dtype=np.int32), 0, status, np.inf)

    if not 0 <= n_drafts <= K:
        return bad(BADPARAM)
    if any(not 0 <= x < V for x in drafts[:n_drafts]):
        return bad(BADTOKEN)
    kept, refused = 0, False
    seen = []
    for j in range(n_drafts):
        x, u = int(drafts[j]), float(accept_u[j])
        px, qx = float(p[j, x]), 1.0 if q is None else float(q[j, x])
        seen.append((px, qx, u))
        if not u * qx < px:
            refused = True
            break
        kept += 1
    if not all(_is_probability(px) and _is_probability(qx) for px, qx, _ in seen):
        return bad(NONFINITE)
    if not all(0 <= u < 1 for _, _, u in seen) or not 0 <= draw_u < 1:
        return bad(BADPARAM)
    w = p[kept].copy()
    if not _is_probability(w).all():
        return bad(NONFINITE)
    if refused:
        if q is None:
            w[int(drafts[kept])] -= 1.0
        else:
            less = np.asarray(q[kept], dtype=np.float64)
            if not _is_probability(less).all():
                return bad(NONFINITE)
            w = w - less
        w = np.maximum(w, 0.0)
        if w.sum() == 0:
            w = p[kept]
    c = np.cumsum(w)
    if c[-1] == 0:
        return bad(EMPTY)
    aim = float(draw_u) * c[-1]
    above = np.nonzero(c > aim)[0]
    token = int(above[0]) if above.size else int(np.nonzero(w)[0][-1])
    out = np.full(K + 1, -1, dtype=np.int32)
    out[:kept] = drafts[:kept]
    out[kept] = token
    return Result(out, kept, OK, float(np.abs(c - aim).min() / c[-1]))
