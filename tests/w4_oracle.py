"""Plain 64-bit forms of 4-bit weights and their products, and error bounds
that the kernels' arithmetic allows (shared by the tests of those operators).

Every fp32 addition or product is taken as off by at most 2^-23 of its result
(the matrix cores need not round to nearest)."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
ULP = 2.0 ** -23


def random_weights(rng, groups, n, k, fmt, group, zeros):
    """codes [groups][n][k/2] uint8, scales (E8M0 bytes, or fp32 values that
    bf16 and fp16 hold), zero points or None."""
    codes = rng.integers(0, 256, (groups, n, k // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        scales = rng.integers(115, 135, (groups, n, k // group)).astype(np.uint8)
    else:
        scales = np.ldexp(rng.integers(128, 256, (groups, n, k // group)) / 256.0,
                          rng.integers(-6, 1, (groups, n, k // group))).astype(np.float32)
        scales *= rng.choice([-1, 1], scales.shape)
    z = rng.integers(0, 16, (groups, n, k // group)).astype(np.uint8) if zeros else None
    return codes, scales, z


def nibbles(codes):
    out = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), np.int64)
    out[..., 0::2], out[..., 1::2] = codes & 15, codes >> 4
    return out


def values(codes, scales, zeros, fmt, group):
    """fp64 weights [groups][n][k], and the same shape of |scale| per value."""
    q = nibbles(codes)
    if fmt == "mxfp4":
        s = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), group, -1)
        return E2M1[q] * s, s
    s = np.repeat(scales.astype(np.float64), group, -1)
    z = 8 if zeros is None else np.repeat(zeros.astype(int), group, -1)
    return (q - z) * s, np.abs(s)


def product(x, w, sabs, fmt, group):
    """x [M][k], w [n][k] -> (y, bound on the fp32 sums' error).

    MXFP4: a 32-wide matrix step is taken to round the running sum eight times
    (at most ULP of a partial sum that the absolute sum bounds), so k / 4 times
    in all, and the waves' sums are added.  INT4: the
    partial sums of a group hold x (16 + q) and the offset, at most 31 + 31
    |x|, `group` terms of them; then k / group scaled groups are added."""
    y = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    k = x.shape[1]
    if fmt == "mxfp4":
        return y, (k / 4 + 40) * ULP * mag
    return y, (group + 4) * ULP * 62 * (np.abs(x) @ sabs.T) + (k / group + 40) * ULP * mag


def rounded(y, bound):
    """Total bound of a bf16 output: the sums' and half a step of bf16."""
    return bound + (np.abs(y) + bound) * 2.0 ** -8 + 2.0 ** -133


def silu(z):
    return z / (1 + np.exp(-z))


def expert(x, gate, up, down, fmt, group):
    """One expert's rows in 64 bits, the bound of the error that reaches them
    through the hidden values, and the absolute sums of the last product (and
    of |a| |scale|, for INT4's offset).  gate, up, down: (w, sabs) pairs.
    d silu / dz lies in [-0.1, 1.1]; silu's own evaluation is taken as off by
    2^-20 (1 + |z|) of its value; a (times its weight) is rounded to bf16."""
    g, dg = product(x, *gate, fmt, group)
    u, du = product(x, *up, fmt, group)
    a = silu(g) * u
    da = 1.1 * dg * (np.abs(u) + du) + np.abs(silu(g)) * du + 2.0 ** -20 * (1 + np.abs(g)) * np.abs(a)
    da = da + (np.abs(a) + da) * (2.0 ** -8 + 4 * ULP)
    return (a @ down[0].T, da @ np.abs(down[0]).T, (np.abs(a) + da) @ np.abs(down[0]).T,
            (np.abs(a) + da) @ down[1].T)


def layer(x, idx, wt, experts, first, fmt, group, shared=None):
    """experts: per expert (gate, up, down) pairs.  Returns (out, bound).  The
    experts' products accumulate in one sum: every rounding of the running sum
    is bounded by ULP of the absolute sum over all of them."""
    T, k = idx.shape
    n, K = experts[0][2][0].shape
    out, through, mag, off = (np.zeros((T, n)) for _ in range(4))

    def add(t, w, mats):
        y, d, a, s = expert(x[t], *mats, fmt, group)
        for to, v in ((out, w * y), (through, np.abs(w) * d), (mag, np.abs(w) * a),
                      (off, np.abs(w) * s)):
            np.add.at(to, t, v)

    for e, mats in enumerate(experts):
        t, j = np.nonzero(idx.astype(np.int64) - first == e)
        if len(t):
            add(t, wt[t, j][:, None].astype(np.float64), mats)
    terms = k * K
    if shared is not None:
        add(np.arange(T), np.ones((T, 1)), shared)
        terms += shared[2][0].shape[1]
    if fmt == "mxfp4":
        sums = (terms / 4 + 40) * ULP * mag
    else:
        sums = (group + 4) * ULP * 62 * off + (terms / group + 40) * ULP * mag
    return out, rounded(out, through + sums)
