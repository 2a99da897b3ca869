"""float64 oracle of the mixture-of-experts layer, written from its definition
(a loop over tokens and choices):

    y[t] = sum_j w[t, j] D_e (act(G_e x[t]) * (U_e x[t])),   e = ids[t, j]

and a bound of what float32 arithmetic may be off by.
"""
from __future__ import annotations

import numpy as np

from .w4_ref import w4_apply_ref, w4_magnitude_ref


def act_ref(kind: str, g):
    g = np.asarray(g, np.float64)
    if kind == "silu":
        return g / (1 + np.exp(-g))
    return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def _named(m, e):
    packed, scales, zeros = m
    return packed[e], scales[e], None if zeros is None else zeros[e]


def moe_ref(gate, up, down, group, group_down, x, ids, weights, act="silu", h_bits=None):
    """(y, bound) [T, d_out]: y, and what y may be off by before its own
    rounding.  A matrix is (codes, scales, zeros or None), a stack of experts.

    The bound.  A product's float32 sums are off by at most steps 2^-23 of the
    magnitudes added up (w4_magnitude_ref; steps: the additions of a group, of
    the groups and of the waves).  |act'| stays below 1.13.  act itself is a few
    float32 steps, of which the argument of exp carries 4 (gelu), times that
    argument: (8 + 6 |v|) 2^-24.  h is then held to h_bits bits (None: in whole).
    What h is off by passes through |D|; the weighted sum adds k + 32 steps."""
    T, k = ids.shape
    n, d_out = down[0].shape[:2]
    x = np.asarray(x, np.float64)
    y, bound = np.zeros((T, d_out)), np.zeros((T, d_out))
    def steps(d, g):
        gran = min(128, g)
        return (gran + -(-d // gran) + 32) * 2.0 ** -23
    d, ffn = x.shape[1], gate[0].shape[1]
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if not 0 <= e < n:
                continue
            w = float(weights[t, j])
            G, U, D = _named(gate, e), _named(up, e), _named(down, e)
            g, u = w4_apply_ref(*G, group, x[t: t + 1])[0], w4_apply_ref(*U, group, x[t: t + 1])[0]
            dg = steps(d, group) * w4_magnitude_ref(*G, group, x[t: t + 1])[0]
            du = steps(d, group) * w4_magnitude_ref(*U, group, x[t: t + 1])[0]
            a = act_ref(act, g)
            h = a * u
            v = np.abs(g) if act == "silu" else 1.6 * (np.abs(g) + 0.045 * np.abs(g) ** 3)
            dh = 1.13 * np.abs(u) * dg + np.abs(a) * du + 1.13 * dg * du + (9 + 6 * v) * 2.0 ** -24 * np.abs(h)
            if h_bits is not None:
                dh = dh + 2.0 ** -h_bits * (np.abs(h) + dh)
            out = w4_apply_ref(*D, group_down, h[None])[0]
            y[t] += w * out
            mag = w4_magnitude_ref(*D, group_down, (np.abs(h) + dh)[None])[0] * 1.01
            through = np.abs(w4_apply_abs(*D, group_down, dh))
            bound[t] += abs(w) * (through + (steps(ffn, group_down) + (k + 32) * 2.0 ** -24) * mag)
    return y, bound


def w4_apply_abs(packed, scales, zeros, group, v):
    """|W| v of a vector v >= 0."""
    from .w4_ref import w4_matrix_ref

    return np.abs(w4_matrix_ref(packed, scales, zeros, group)) @ v
