"""Layers of experts whose exact outputs float32 holds, so that a kernel that
loses a bit, an input or a feature on the way is seen in the output's bits.

Features come in pairs.  The gate of every feature is 64 (one input is 1, its
weight 64), where silu and gelu are the identity in float32: exp(-64) is lost
beside 1.  Up takes one input or two, and down one pair or one feature for each
output; all other weights are 0 (the code is the zero point).

bf16 rows.  x holds +-(1 + m / 128).  The features of a pair are
    u = x[k1] + 2^-8 x[k2],   u' = x[k1] + 2^-8 x[k2'],
16 bits each, and an output is a sum of 64 (u - u') = 2^-2 (x[k2] - x[k2']): the
upper 8 bits of h cancel, its lower ones remain.  Every sum on the way is exact:
a group of 128 products of (32 + q) <= 47 with x is below 2^14 in steps of 2^-7,
21 bits; with the upper parts of h (steps of 1/4, below 2^7) and the lower ones
(steps of 2^-9, below 1/2) 22 and 21 bits.  The weights are 1/2, 1 or 2, and the
32 choices' sum takes 16 bits.  Where one group holds all inputs, u = x[k1] and
u' = x[k1'].

float32 rows.  x holds 24 bits of any size, u = x[k1], and an output is the sum of
one feature of each choice, 24 bits each: one choice is exact, and the sum of k
rounds k - 1 times.
"""
from __future__ import annotations

import numpy as np

ONE = 64.0  # the gate


class Matrices:
    """A stack of matrices of zeros, to be given some weights q - z."""

    def __init__(self, rng, n, d_out, d_in, group, zeros):
        self.group = group
        shape = (n, d_out, -(-d_in // group))
        self.zeros = rng.integers(1, 15, shape).astype(np.uint8) if zeros else None
        z = np.full(shape, 8, np.uint8) if self.zeros is None else self.zeros
        self.codes = np.ascontiguousarray(np.repeat(z, group, 2)[..., :d_in])
        self.scales = np.ones(shape, np.float32)

    def put(self, e, o, k, weight, scale=1.0):
        self.codes[e, o, k] += np.asarray(weight, np.int64).astype(np.uint8)
        self.scales[e, o, k // self.group] = scale

    def packed(self):
        """(codes, scales, zeros) as a checkpoint holds them."""
        assert self.codes.max() < 16
        return self.codes[..., 0::2] | (self.codes[..., 1::2] << 4), self.scales, self.zeros


class ExactLayer:
    def __init__(self, seed, n, d, ffn, d_out, group, zeros, dtype, group_down=None):
        rng = np.random.default_rng(seed)
        self.n, self.d, self.ffn, self.d_out, self.dtype = n, d, ffn, d_out, dtype
        self.gate = Matrices(rng, n, ffn, d, group, zeros)
        self.up = Matrices(rng, n, ffn, d, group, zeros)
        self.down = Matrices(rng, n, d_out, ffn, group_down or group, zeros)
        self.one = d // 2  # the input that is 1
        self.two = dtype == "bf16" and d > group  # two inputs to a feature
        pairs = ffn // 2
        f = np.arange(ffn)
        e, f2 = np.arange(n)[:, None], f[None, :]
        self.gate.put(e, f2, self.one, 1, ONE)
        # The last features take the last inputs.
        last = (d - 1 - (pairs - 1 - f // 2) * 7) % d
        if self.two:
            groups = -(-d // group)
            g1 = (last // group + 1) % groups  # the group of the first input is another one
            first = g1 * group + f // 2 % np.minimum(group, d - g1 * group)
            other = rng.integers(0, d, (n, ffn))
            other = np.where(f % 2 == 0, last, np.where(other // group == g1, last ^ 1, other))
            assert (other // group != first // group).all()
        else:
            first = (d - 1 - (ffn - 1 - f) * 7) % d
        self.k1 = np.broadcast_to(first, (n, ffn))
        self.sign = np.repeat(rng.choice([-1, 1], (n, pairs)), 2, 1)
        self.up.put(e, f2, self.k1, self.sign)
        if self.two:
            self.k2 = other
            self.up.put(e, f2, self.k2, 1, 2.0 ** -8)
        # The first outputs take the last features; the experts go on where the one before ends.
        o = np.arange(d_out)
        if dtype == "bf16":
            p = (pairs - 1 - (o[None, :] + np.arange(n)[:, None] * d_out)) % pairs
            self.f1, self.f2 = 2 * p, 2 * p + 1
            self.down.put(e, o[None, :], self.f1, 1)
            self.down.put(e, o[None, :], self.f2, -1)
        else:
            self.f1 = (ffn - 1 - (o[None, :] + np.arange(n)[:, None] * d_out)) % ffn
            self.f2 = None
            self.down.put(e, o[None, :], self.f1, 1)

    def inputs(self, seed, T, k):
        """x, ids and weights; every seventh choice names no expert, and the first
        token's first is expert 0."""
        rng = np.random.default_rng(seed)
        if self.dtype == "bf16":
            x = rng.choice([-1.0, 1.0], (T, self.d)) * (1 + rng.integers(0, 128, (T, self.d)) / 128)
        else:
            x = rng.choice([-1.0, 1.0], (T, self.d)) * rng.uniform(1, 2, (T, self.d)) * 2.0 ** rng.integers(-3, 4, (T, self.d))
        x[:, self.one] = 1.0
        ids = np.argsort(rng.random((T, self.n)), 1)[:, :k].astype(np.int32)
        if ids[0, 0] != 0:
            ids[0][ids[0] == 0] = ids[0, 0]
            ids[0, 0] = 0
        absent = np.arange(T * k).reshape(T, k) % 7 == 6
        ids = np.where(absent, np.where(absent.cumsum(1) % 2 == 1, -1, self.n), ids).astype(np.int32)
        return x.astype(np.float32), np.ascontiguousarray(ids), rng.choice([0.5, 1.0, 2.0], (T, k)).astype(np.float32)

    def h(self, x, e, keep_x=None):
        """act(G_e x) (U_e x) in float64 of rows x; keep_x: bits of x, the others cut."""
        v = cut(x, keep_x) if keep_x else np.asarray(x, np.float64)
        u = self.sign[e] * v[:, self.k1[e]]
        if self.two:
            u = u + 2.0 ** -8 * v[:, self.k2[e]]
        return ONE * u

    def ref(self, x, ids, w, *, keep_x=None, keep_h=None, features=None, inputs=None):
        """(y, sum of the absolute values of its terms), float64.  The rest are
        faults: bits of x or of h that are kept, features or inputs of which
        only the first are taken."""
        x = np.asarray(x, np.float64)
        if inputs is not None:
            x = np.where(np.arange(self.d) < inputs, x, 0.0)
        y, mag = np.zeros((x.shape[0], self.d_out)), np.zeros((x.shape[0], self.d_out))
        for e in range(self.n):
            t, j = np.nonzero(ids == e)
            if t.size == 0:
                continue
            h = self.h(x[t], e, keep_x)
            if keep_h:
                h = cut(h, keep_h)
            if features is not None:
                h = np.where(np.arange(self.ffn) < features, h, 0.0)
            v = h[:, self.f1[e]] - (h[:, self.f2[e]] if self.f2 is not None else 0.0)
            v = v * w[t, j].astype(np.float64)[:, None]
            np.add.at(y, t, v)
            np.add.at(mag, t, np.abs(v))
        return y, mag


def cut(v, bits):
    """v with its first `bits` significant bits."""
    m, e = np.frexp(np.asarray(v, np.float64))
    return np.ldexp(np.trunc(m * 2.0 ** bits) / 2.0 ** bits, e)


class ActLayer:
    """One feature for each output: gate (q - z) / 2 x[k], up 1, down 1, so that y
    is w act(g) with g known to float32's last bits.  Only every eighth feature has
    a gate, and the scales of down's groups without a weight are 0, so that little
    else is added to an output."""

    def __init__(self, seed, n, d, ffn, d_out, group, zeros):
        rng = np.random.default_rng(seed)
        self.n, self.d, self.ffn, self.d_out, self.one = n, d, ffn, d_out, d // 2
        self.gate = Matrices(rng, n, ffn, d, group, zeros)
        self.up = Matrices(rng, n, ffn, d, group, zeros)
        self.down = Matrices(rng, n, d_out, ffn, 32, zeros)
        e, f = np.arange(n)[:, None], np.arange(ffn)[None, :]
        self.k = rng.integers(0, d, (n, ffn))
        z = np.full(self.gate.scales.shape, 8) if self.gate.zeros is None else self.gate.zeros
        at = z[e, f, self.k // group].astype(np.int64)
        self.weight = np.clip(rng.integers(1, 5, (n, ffn)) * rng.choice([-1, 1], (n, ffn)), -at, 15 - at)  # q - z
        i = np.arange(ffn // 8)
        used = 8 * i + 3 * i % 8
        self.weight[:, np.isin(f[0], used, invert=True)] = 0
        self.gate.put(e, f, self.k, self.weight, 0.5)
        self.up.put(e, f, self.one, 1)
        o = np.arange(d_out)[None, :]
        self.f = used[(used.size - 1 - (o + np.arange(n)[:, None] * d_out)) % used.size]
        self.down.scales[:] = 0
        self.down.put(e, o, self.f, 1)

    def gates(self, x, e):
        return 0.5 * self.weight[e] * np.asarray(x, np.float64)[:, self.k[e]]
