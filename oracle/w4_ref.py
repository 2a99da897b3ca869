"""float64 oracle of the 4-bit base products and of the router, written from
the definitions (loops over groups, experts and choices; no code shared with
the HIP path).

    W[o, k] = s[o, k // G] (q[o, k] - z[o, k // G]),  z = 8 without zero points
"""
from __future__ import annotations

import math

import numpy as np


def unpack_ref(packed: np.ndarray) -> np.ndarray:
    """Codes [..., d_in] of bytes [..., d_in / 2]: input 2 i in the low four bits."""
    out = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), np.int64)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def w4_matrix_ref(packed, scales, zeros, group: int) -> np.ndarray:
    """One matrix in float64."""
    q = unpack_ref(packed)
    w = np.empty(q.shape, np.float64)
    for g in range(scales.shape[-1]):
        at = slice(g * group, min(q.shape[-1], (g + 1) * group))
        z = 8 if zeros is None else zeros[..., g: g + 1].astype(np.int64)
        w[..., at] = (q[..., at] - z) * scales[..., g: g + 1].astype(np.float64)
    return w


def w4_apply_ref(packed, scales, zeros, group: int, x) -> np.ndarray:
    return np.asarray(x, np.float64) @ w4_matrix_ref(packed, scales, zeros, group).T


def w4_magnitude_ref(packed, scales, zeros, group: int, x) -> np.ndarray:
    """sum_k |s| (32 + q + 32 + z) |x|: what the products and their correction
    add up to in absolute value, the measure of a float32 sum's error."""
    q = unpack_ref(packed)
    m = np.empty(q.shape, np.float64)
    for g in range(scales.shape[-1]):
        at = slice(g * group, min(q.shape[-1], (g + 1) * group))
        z = 8 if zeros is None else zeros[..., g: g + 1].astype(np.int64)
        m[..., at] = (64 + q[..., at] + z) * np.abs(scales[..., g: g + 1].astype(np.float64))
    return np.abs(np.asarray(x, np.float64)) @ m.T


def experts_ref(packed, scales, zeros, group: int, x, ids, weights=None, product=w4_apply_ref):
    """Rows [T k, d_out] (zero without an expert), or with weights [T, d_out]."""
    T, k = ids.shape
    n, d_out = packed.shape[:2]
    rows = np.zeros((T * k, d_out))
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if 0 <= e < n:
                xr = x[t * k + j] if x.shape[0] == T * k else x[t]
                rows[t * k + j] = product(packed[e], scales[e], None if zeros is None else zeros[e], group, xr[None])[0]
    if weights is None:
        return rows
    y = np.zeros((T, d_out))
    for t in range(T):
        for j in range(k):
            if 0 <= int(ids[t, j]) < n:
                y[t] += float(weights[t, j]) * rows[t * k + j]
    return y


def pair_order(a: float, b: float):
    """A key that orders as sigmoid(a) + sigmoid(b) does; -inf stands for no
    logit, and sums without two come first.  The sum is held as it is, or as
    its distance from one or two where it is near them, which a float holds
    where 1 - 2^-60 is not one."""
    hi, lo = max(a, b), min(a, b)
    if lo == -math.inf:
        return (-1, 0.0)
    p, q = (math.exp(-abs(v)) / (1 + math.exp(-abs(v))) for v in (hi, lo))
    if hi <= 0:
        return (0, p + q) if p + q < 0.5 else (1, p + q - 1)
    if lo >= 0:
        return (2, -(p + q)) if p + q < 0.5 else (1, 1 - (p + q))
    return (1, q - p)


def route_ref(logits, k: int, *, score="softmax", bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """(ids [T, k], weights [T, k] float64), one token at a time."""
    T, E = logits.shape
    n = E // groups
    fmax = float(np.finfo(np.float32).max)
    ids = np.full((T, k), -1, np.int64)
    weights = np.zeros((T, k))
    for t in range(T):
        l = [min(float(v), fmax) if v == v else -math.inf for v in logits[t]]
        if score == "softmax":
            top = max(l)
            ex = [math.exp(v - top) if v > -math.inf else 0.0 for v in l]
            s = [v / math.fsum(ex) if v else 0.0 for v in ex]
        else:
            s = [0.0 if v == -math.inf else (1 / (1 + math.exp(-v)) if v > 0 else math.exp(v) / (1 + math.exp(v)))
                 for v in l]
        # Without a bias the order of c is the order of the logits, which no
        # rounding of exp can make equal.
        if bias is None:
            c = list(l)
        else:
            c = [a + min(float(b), fmax) for a, b in zip(s, bias)]
        c = [-math.inf if l[e] == -math.inf or c[e] != c[e] else c[e] for e in range(E)]
        if groups > 1:
            of = []
            for g in range(groups):
                part = range(g * n, (g + 1) * n)
                if score == "softmax" or n == 1:
                    of.append(max(c[e] for e in part))
                else:
                    two = sorted((c[e] for e in part), reverse=True)[:2]
                    of.append(two[0] + two[1] if bias is not None else pair_order(*two))
            keep = sorted(range(groups), key=lambda g: of[g], reverse=True)[:top_groups]  # stable: ties to the lowest
            c = [c[e] if e // n in keep else -math.inf for e in range(E)]
        order = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > -math.inf][:k]
        w = [s[e] for e in order]
        if renormalize and order:
            if score == "softmax" or not any(w):  # the ratios, where the scores themselves are below any number
                hi = max(l[e] for e in order)
                w = [math.exp(l[e] - hi) for e in order]
            total = math.fsum(w)
            w = [v / total for v in w]
        for j, e in enumerate(order):
            ids[t, j], weights[t, j] = e, w[j] * scale
    return ids, weights
