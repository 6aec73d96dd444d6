"""Plain reference of the 8-bit output projection: row codes and their product.

quantize_rows [P1 "int8 weights": per-row absmax]: the scale of a row is
max |x| times 1/127, in float32; a code is the quotient by that float32 scale,
to the nearest whole number (ties to even), held to [-127, 127]. Formed in
float64, which holds every quotient of two float32 values far enough from a
half that is not one: with |code| <= 127 a quotient other than a half differs
from it by more than 2^-33 relative.

int8_logits: the sum in whole numbers, the scales and the bias in float64.
"""
from __future__ import annotations

import numpy as np


def quantize_rows(x):
    """x [rows, width] float32 values -> (codes int8, scale float32)."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    codes = np.zeros(x.shape, dtype=np.int8)
    scale = np.zeros(x.shape[0], dtype=np.float32)
    for r, row in enumerate(x):
        if not np.isfinite(row).all():
            scale[r] = np.nan
            continue
        s = np.float32(np.abs(row).max()) * (np.float32(1.0) / np.float32(127.0))
        scale[r] = s
        if s > 0:
            codes[r] = np.clip(np.rint(row / np.float64(s)), -127, 127)
    return codes, scale


def int8_logits(codes, code_scale, weight, w_scale, bias=None):
    """-> (logits float64 [rows, vocab], |sum| * scales, the products' size)."""
    acc = codes.astype(np.int64) @ weight.astype(np.int64).T
    v = acc.astype(np.float64) * code_scale.astype(np.float64)[:, None] * \
        w_scale.astype(np.float64)
    out = v if bias is None else v + bias.astype(np.float64)
    return out, np.abs(v)


def logits_bound(out, product, dtype):
    """How far int8_logits may be from `out`: the sum rounded to float32 and its
    product with the row's scale rounded (2^-24 each, relative to the product),
    the fma's rounding (2^-24 of the result), and for bfloat16 the rounding to
    it (2^-8 of the float32 result)."""
    b = 2.0 ** -23 * product + 2.0 ** -24 * np.abs(out)
    if dtype == "bf16":
        b = b + 2.0 ** -8 * (np.abs(out) + b)
    return b * (1 + 2.0 ** -20) + 1e-44   # second order; results below the normal range
