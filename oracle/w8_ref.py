"""Oracle of the 8-bit base products, written from the definitions (integers
and float64; no code shared with the HIP path).

    scales[t] = a / 127,  q[t, k] = nearest(127 x[t, k] / a),  a = max |x[t]|
    y[t, o] = s_x[t] s_w[o] sum_k q_x[t, k] q_w[o, k]
"""
from __future__ import annotations

import numpy as np


def w8_quantize_ref(x):
    """(codes int64 [T, d], scales float64 [T]) of float32 values.  Whether x
    lies above the border between k and k + 1 is the sign of 254 |x| - (2 k +
    1) a, both of which float64 holds exactly; on it the even one is taken."""
    x = np.asarray(x, np.float32).astype(np.float64)
    codes, scales = np.zeros(x.shape, np.int64), np.zeros(x.shape[0])
    for t in range(x.shape[0]):
        v = np.abs(x[t])
        if not np.isfinite(v).all():
            scales[t] = np.nan
            continue
        a = v.max(initial=0.0)
        scales[t] = a / 127
        if a == 0:
            continue
        k = np.zeros(v.shape, np.int64)
        for n in range(127):  # the codes are counted up, border by border
            over = 254 * v - (2 * n + 1) * a
            k += (over > 0) | ((over == 0) & (n % 2 == 1))
        codes[t] = np.where(x[t] < 0, -k, k)
    return codes, scales


def w8_product_ref(q, s, w, sw):
    """y in float64, from integer sums."""
    total = np.asarray(q, np.int64) @ np.asarray(w, np.int64).T
    return total * np.asarray(s, np.float64)[:, None] * np.asarray(sw, np.float64)[None, :]


def w8_apply_ref(x, w, sw):
    return w8_product_ref(*w8_quantize_ref(x), w, sw)
