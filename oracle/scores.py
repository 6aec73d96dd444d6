"""Plain references of the calls around the logits: the RMS norm with a residual and
8-bit codes, log probabilities with entropy and the likeliest ids, their gradient, and
distillation from a teacher's top entries; each with the bound that the kernels'
roundings keep.

Everything is formed in float64 (codes in numpy's long double, whose 64-bit
mantissa holds 127 times a product of two float32 values exactly and a quotient far
enough from a half that is not one).

Bounds count roundings of u = 2^-24 relative (float32, half a step). A weight
e_j = 2^x_j, x_j = (z_j - M) log2(e) / T, has a difference, a constant and a product
rounded (3 u |x_j|, so 3 ln 2 u |x_j| of e_j) and an exponential good to 2 u; a sum
adds at most 16 float32 terms before it goes on in 64 bits (15 u). ``weight_error``
is that sum's relative error, with m = sum_j p_j |x_j|: (2.1 m + 18) u.

The hardware's exponential gives 0 where 2^x is below the smallest normal number,
so a weight may be off by 2^-126 (``TINY`` is twice that), and a gradient's element by
that times the row's factor. Sums hold a weight of 1, the largest's, and do not feel it.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
LN2 = float(np.log(2.0))
REST_MIN = 2.0 ** -20
TINY = 2.0 ** -125
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def round_bf16(x):
    """float32 values rounded to bfloat16, ties to even, as float32."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x), r, x).astype(np.float32)


def norm_quantize(x, weight=None, eps=1e-6, residual=None, dtype="f32"):
    """float32 values -> (codes int8, scale float64, h float32)."""
    with np.errstate(all="ignore"):
        h = np.asarray(x, dtype=np.float32)
        if residual is not None:
            h = h + np.asarray(residual, dtype=np.float32)
            h = round_bf16(h) if dtype == "bf16" else h
        rows, width = h.shape
        w = np.ones(width) if weight is None else np.asarray(weight, dtype=np.float64)
        t = h.astype(np.float64) * w
        codes = np.zeros(h.shape, dtype=np.int8)
        scale = np.zeros(rows)
        for r in range(rows):
            if not (np.isfinite(h[r]).all() and np.isfinite(t[r]).all()):
                scale[r] = np.nan
                continue
            m = np.abs(t[r]).max()
            if m == 0:
                continue
            scale[r] = m / (127 * np.sqrt((h[r].astype(np.float64) ** 2).mean() + eps))
            codes[r] = np.rint(t[r].astype(np.longdouble) * 127 / np.longdouble(m)).astype(np.int8)
    return codes, scale, h


def row_state(z):
    """0, 1 (a NaN or +inf) or 2 (all -inf)."""
    if np.isnan(z).any() or (z == np.inf).any():
        return 1
    return 2 if (z == -np.inf).all() else 0


def exponents(z, T):
    """z - M over T, in units of log 2; M."""
    M = z.max()
    return (z - M) / T / LN2, M


def weight_error(p, x):
    fin = p > 0
    return (2.1 * float((p[fin] * np.abs(x[fin])).sum()) + 18.0) * U


def logprobs(z, tokens, k, T=1.0):
    """One row -> a dict of its outputs and of their bounds (under "off")."""
    z = np.asarray(z, dtype=np.float64)
    n, V = len(tokens), len(z)
    st = row_state(z)
    bad = any(t != -1 and not 0 <= t < V for t in tokens)
    out = dict(status=st if st else 3 if bad else 0)
    if st:
        out.update(logprob=np.array([0.0 if t == -1 else np.nan for t in tokens]), entropy=np.nan,
                   top_ids=np.full(k, -1), top_logprob=np.full(k, np.nan),
                   norm=np.full(2, np.nan))
        out["off"] = dict(logprob=np.zeros(n), entropy=0.0, top_logprob=np.zeros(k),
                          norm=np.zeros(2))
        return out
    x, M = exponents(z, T)
    e = np.exp2(x)
    Z = e.sum()
    p = e / Z
    fin = p > 0
    m1 = float((p[fin] * np.abs(x[fin])).sum())
    m2 = float((p[fin] * x[fin] ** 2).sum())
    zerr = weight_error(p, x)

    def lp(v):   # results are float32: -inf past its range
        y = (v - M) / T - np.log(Z)
        return np.where(y < -3.4028235677973366e38, -np.inf, y)

    got = np.array([0.0 if t == -1 else lp(z[t]) if 0 <= t < V else np.nan for t in tokens])
    order = np.argsort(-z, kind="stable")[:k]
    ids, top = np.full(k, -1), np.full(k, -np.inf)
    real = order[z[order] > -np.inf]
    ids[:len(real)], top[:len(real)] = real, lp(z[real])
    out.update(logprob=got, entropy=np.log(Z) + LN2 * m1, top_ids=ids, top_logprob=top,
               norm=np.array([M, Z]))

    def around(v):   # the sum's error, and one rounding of the result
        return zerr + U * np.where(np.isfinite(v), np.abs(v), 0.0) + 1e-40

    # entropy: e x has its weight's error and a product's; the quotient the sum's
    H = out["entropy"]
    off_h = U * LN2 * (2.1 * m2 + 20 * m1) + (LN2 * m1 + 1) * zerr + U * H + 1e-40
    out["off"] = dict(logprob=around(got), entropy=off_h, top_logprob=around(top),
                      norm=np.array([0.0, (zerr + U) * Z]))
    return out


def logprobs_grad(z, tokens, norm, g, T=1.0, H=0.0, ge=0.0, dtype="f32"):
    """One row -> (gradient, how far off it may be), from the norm and entropy given."""
    z = np.asarray(z, dtype=np.float64)
    V = len(z)
    real = [(t, float(gi)) for t, gi in zip(tokens, g) if t != -1]
    if any(not 0 <= t < V for t, _ in real):
        return np.full(V, np.nan), np.zeros(V)
    if not any(gi for _, gi in real) and ge == 0.0:
        return np.zeros(V), np.zeros(V)
    M, Z = float(norm[0]), float(norm[1])
    x = (z - M) / T / LN2
    p = np.exp2(x) / Z
    logp = np.where(p > 0, np.where(np.isfinite(x), x, 0.0) * LN2 - np.log(Z), 0.0)
    G = sum(gi for _, gi in real)
    out = -p * (G + ge * (logp + H))
    size = p * (abs(G) + abs(ge) * (np.abs(logp) + 2 * np.log(Z) + abs(H)))
    ax = np.where(p > 0, np.abs(np.where(np.isfinite(x), x, 0.0)), 0.0)
    off = size * (2.1 * ax + 12.0) * U
    # an exponent may be formed as z c - fl(M c), with what the rounding of M c leaves, at
    # most u |M c|, put back through a factor that is itself rounded (twice, u each)
    off += p * abs(ge) * 4 * U * U * abs(M / T / LN2)
    for t, gi in real:
        out[t] += gi
        off[t] += abs(gi) * len(real) * 2.0 ** -52   # their sum in 64 bits
    for t in {t for t, _ in real}:
        off[t] += U * abs(out[t])   # with the id's own weight, rounded to float32 first
    off += TINY * (abs(G) + abs(ge) * (88 + 2 * np.log(Z) + abs(H)))
    out, off = out / T, off / T * (1 + 4 * U)
    return out, off + HALF_STEP[dtype] * (np.abs(out) + off) + TINY


def distill(z, ids, teacher, T=1.0, tail=False, weight=1.0, dtype="f32"):
    """One row -> dict(loss, grad, status, off_loss, off_grad)."""
    z = np.asarray(z, dtype=np.float64)
    t = np.asarray(teacher, dtype=np.float32).astype(np.float64)
    V = len(z)
    zero = np.zeros(V)
    if weight == 0.0:
        return dict(loss=0.0, grad=zero, status=0, off_loss=0.0, off_grad=zero)
    real = [i for i, j in enumerate(ids) if j != -1]
    status = 0
    if any(not 0 <= ids[i] < V for i in real):
        status = 3
    elif any(not t[i] < np.inf for i in real):
        status = 1
    elif not any(t[i] > -np.inf for i in real):
        status = 2
    status = status or row_state(z)
    if status:
        return dict(loss=np.nan, grad=np.full(V, np.nan), status=status, off_loss=0.0,
                    off_grad=zero)
    with np.errstate(all="ignore"):
        q = {i: np.exp(t[i]) if tail else np.exp(t[i] - max(t[j] for j in real)) for i in real}
        total = sum(q.values())
        rest = 0.0
        if tail:
            rest = 1.0 - total
            rest = rest if rest > REST_MIN else 0.0
        else:
            q = {i: v / total for i, v in q.items()}
        x, M = exponents(z, T)
        e = np.exp2(x)
        inside = np.zeros(V, dtype=bool)
        inside[[ids[i] for i in real]] = True
        Z = e.sum()
        p = e / Z
        logp = (z - M) / T - np.log(Z)
        zerr = weight_error(p, x)
        # the other ids against their own largest, however far below M it is
        log_pr, share, rerr = -np.inf, np.zeros(V), 0.0
        if (z[~inside] > -np.inf).any():
            xr, Mr = exponents(np.where(inside, -np.inf, z), T)
            er = np.exp2(xr)
            log_pr = np.log(er.sum()) + (Mr - M) / T - np.log(Z)
            share = er / er.sum()
            rerr = weight_error(share, xr)
        loss, off = 0.0, 0.0
        for i in real:
            if q[i] > 0:
                loss += q[i] * (np.log(q[i]) - logp[ids[i]])
                off += q[i] * zerr
        if rest > 0:
            loss += rest * (np.log(rest) - log_pr)
            off += rest * (zerr + rerr)
        whole = sum(q.values()) + rest
        grad = p * whole - share * rest
        ax = np.abs(np.where(np.isfinite(x), x, 0.0))
        off_g = np.abs(grad) * (2.1 * ax + 12.0) * U + p * whole * (zerr + rerr) + \
            share * rest * (zerr + rerr) + TINY * (whole + rest)
        grad[inside] = p[inside] * whole
        off_g[inside] = p[inside] * whole * ((2.1 * ax[inside] + 12.0) * U + zerr)
        for i in real:
            grad[ids[i]] -= q[i]
        grad, off_g = grad * weight / T, off_g * abs(weight) / T
        off_g = off_g + HALF_STEP[dtype] * (np.abs(grad) + off_g) + TINY
        loss *= weight
        off = off * abs(weight) + (U * abs(loss) if np.isfinite(loss) else 0.0) + 1e-38
    return dict(loss=loss, grad=grad, status=0, off_loss=off * (1 + 4 * U), off_grad=off_g)
