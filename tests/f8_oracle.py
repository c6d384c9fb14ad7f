"""Plain 64-bit forms of the 8-bit products with a scale per block of 128, and error
bounds that the kernels' arithmetic allows (shared by the tests of those operators).

Quantising is exact here: the definition names every fp32 rounding.  Every fp32
addition or product after it is taken as off by at most 2^-23 of its result.  The
matrix instruction sums 128 products of codes with their smaller bits cut off below
the largest: with 17 bits kept below the largest product, each of the 128 loses at
most 2^-17 of it, 2^-10 in all."""
from __future__ import annotations

import numpy as np
import torch

B = 128
ULP = 2.0 ** -23
CUT = 2.0 ** -10
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def blocks(a, axis):
    """a with `axis` split into [blocks][128], zeros behind the end."""
    a = np.moveaxis(np.asarray(a), axis, -1)
    pad = [(0, 0)] * (a.ndim - 1) + [(0, -a.shape[-1] % B)]
    a = np.pad(a, pad)
    return a.reshape(*a.shape[:-1], -1, B)


def quantise(x):
    """fp32 x [..][blocks][128] -> (codes uint8, scales [..][blocks]): the documented
    steps in fp32."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        top = np.abs(x).max(-1)
        s = np.maximum(top * np.float32(1 / 448), np.float32(2.0 ** -100))
        inv = np.float32(1) / s
        v = np.clip(x * inv[..., None], np.float32(-448), np.float32(448))
    codes = torch.from_numpy(np.ascontiguousarray(v)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return codes, s


def decode(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()


def rows_quantised(x):
    """(codes, scales, fp64 values [rows][k]) of rows quantised along k."""
    codes, s = quantise(blocks(x, 1))
    v = decode(codes) * s[..., None].astype(np.float64)
    return codes, s, v.reshape(x.shape[0], -1)[:, :x.shape[1]]


def weights_quantised(w):
    """w [groups][k][n] fp32 -> fp64 values [groups][k][n], a scale per 128 x 128."""
    g, k, n = w.shape
    kb, nb = -(-k // B), -(-n // B)
    p = np.zeros((g, kb * B, nb * B), np.float32)
    p[:, :k, :n] = w
    p = p.reshape(g, kb, B, nb, B).transpose(0, 1, 3, 2, 4).reshape(g, kb, nb, B * B)
    codes, s = quantise(p)
    v = decode(codes) * s[..., None].astype(np.float64)
    return v.reshape(g, kb, nb, B, B).transpose(0, 1, 3, 2, 4).reshape(g, kb * B, nb * B)[:, :k, :n]


def random_codes(rng, groups, n, k):
    """Codes [groups][n][k] (no NaN), scales, and their fp64 values [groups][n][k]."""
    codes = rng.integers(0, 256, (groups, n, k), dtype=np.uint8)
    codes[(codes & 127) == 127] = 0
    scales = np.exp(rng.uniform(-8, -6, (groups, -(-n // B), -(-k // B)))).astype(np.float32)
    return codes, scales, weight_values(codes, scales)


def weight_values(codes, scales):
    _, n, k = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), B, 1)[:, :n], B, 2)[:, :, :k]
    return decode(codes) * s


def product(q, w):
    """Rows q [M][k] and weights w [n][k], both fp64 values of codes -> (y, bound of
    the sums' error)."""
    y = q @ w.T
    qm, wm = np.abs(blocks(q, 1)).max(-1), np.abs(blocks(w, 1)).max(-1)
    terms = qm.shape[1] + 24
    return y, CUT * (qm @ wm.T) + terms * ULP * (np.abs(q) @ np.abs(w).T)


def weight_gradient(x, dy):
    """Rows x [M][k] and dy [M][n] of one group, fp32 -> (dw [k][n], bound)."""
    if not len(x):
        z = np.zeros((x.shape[1], dy.shape[1]))
        return z, z
    q = [rows_quantised(np.ascontiguousarray(a.T))[2] for a in (x, dy)]
    return product(q[0], q[1])


def rounded(y, bound, dtype):
    """Total bound of an output of 16 bits: the sums' and half a step of its type."""
    return bound + (np.abs(y) + bound) * HALF[dtype] + LEAST[dtype]
