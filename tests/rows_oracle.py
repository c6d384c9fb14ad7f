"""Plain 64-bit forms of the expert-sorted rows, and the tolerances that the
arithmetic of the kernels allows (shared by the tests of those operators)."""
from __future__ import annotations

import numpy as np


def layout(idx, E, first=0, align=1):
    """counts, offsets, perm (capacity long), inv by the definition, slot by slot."""
    T, k = idx.shape
    slots = [[] for _ in range(E)]
    for f, e in enumerate(int(v) for v in idx.reshape(-1)):
        if 0 <= e - first < E:
            slots[e - first].append(f)
    cap = T * k + min(E, T * k) * (max(align, 1) - 1)
    perm = np.full(cap, -1, np.int32)
    inv = np.full(T * k, -1, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    at = 0
    for e, rows in enumerate(slots):
        for i, f in enumerate(rows):
            perm[at + i], inv[f] = f, at + i
        at += -(-len(rows) // max(align, 1)) * max(align, 1)
        offsets[e + 1] = at
    return np.array([len(r) for r in slots], np.int32), offsets, perm, inv.reshape(T, k)


def padding_rows(counts, offsets):
    return np.concatenate([np.arange(o + c, n) for o, c, n in
                           zip(offsets[:-1], counts, offsets[1:])] or [np.zeros(0, int)]).astype(int)


def unsort(y, w, inv, add=None):
    """(out, bound): the weighted sums in 64 bits, and the sum of the absolute terms."""
    T, k = inv.shape
    out = np.zeros((T, y.shape[1]))
    mag = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0:
                term = (1.0 if w is None else float(w[t, j])) * y[inv[t, j]]
                out[t] += term
                mag[t] += np.abs(term)
    if add is not None:
        out += add
        mag += np.abs(add)
    return out, mag


def unsort_bwd(dout, y, w, inv, rows):
    """dy (zeros where no slot), dw, and the sum of dw's absolute terms."""
    T, k = inv.shape
    dy = np.zeros((rows, dout.shape[1]))
    dw = np.zeros((T, k))
    mag = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = inv[t, j]
            if r >= 0:
                dy[r] = float(w[t, j]) * dout[t]
                dw[t, j] = dout[t] @ y[r]
                mag[t, j] = np.abs(dout[t]) @ np.abs(y[r])
    return dy, dw, mag
