"""float64 products by groups of rows, their gradients, the sum of a token's
results and adapters beside a projection, with the error bounds of a kernel
that sums in fp32 and rounds each result once.

Definitions, for places i of group g (offsets[g] <= i < offsets[g+1]), r_i =
rows[i]:

    D_i  = A_{r_i} B_g^T            dA_i = dD_i B_g      dB_g = sum_i dD_i^T A_{r_i}
    out_t = sum_j w_tj X_{s_tj}     dX_i = (sum_{j: s_tj = i} w_tj) dout_t, t = r_i
                                    dw_tj = dout_t . X_{s_tj}

Arrays are float64; 16-bit values are exact in them.  A bound is the fp32
summation's (each addition off by half a step of the running sum, the
instruction's own additions not better than truncation: twice that, 2 (n + 8)
2^-24 of the sum of the products' magnitudes) and one rounding of the result
to its type.
"""
from __future__ import annotations

import numpy as np

# half a step of the type, relative; half of its smallest step, absolute
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}
F32 = 2.0 ** -24
LOW = 2.0 ** -126       # a product below fp32's least normal may be lost


def group_rows(ids, groups):
    """rows, offsets, slots of ids (tokens,) or (tokens, top), by definition."""
    ids = np.asarray(ids)
    top = ids.shape[1] if ids.ndim == 2 else 1
    flat = ids.reshape(-1)
    places = [[] for _ in range(groups + 1)]
    for c, g in enumerate(flat.tolist()):
        places[g if 0 <= g < groups else groups].append(c)
    order = [c for p in places for c in p]
    offsets = np.cumsum([0] + [len(p) for p in places[:groups]])
    slots = np.full(flat.shape, -1, np.int64)
    for i, c in enumerate(order[:offsets[-1]]):
        slots[c] = i
    return (np.array([c // top for c in order], np.int64), offsets.astype(np.int64),
            slots.reshape(ids.shape))


def _bound(mag, n, want, kind):
    u = UNIT[kind]
    return (1 + u) * 2 * (n + 8) * (F32 * mag + LOW) + u * np.abs(want) + TINY[kind]


def _row(A, rows, i):
    r = i if rows is None else int(rows[i])
    return A[r] if 0 <= r < A.shape[0] else np.zeros(A.shape[1])


def _gather(A, rows, a, b):
    return np.array([_row(A, rows, i) for i in range(a, b)]).reshape(b - a, A.shape[1])


def _spans(offsets, places):
    o = np.clip(offsets, 0, places)
    return [(int(a), max(int(a), int(b))) for a, b in zip(o[:-1], o[1:])]


def product(A, B, offsets, rows, kind):
    """D (NaN in rows of no group) and its bound; kind: D's type."""
    places = A.shape[0] if rows is None else len(rows)
    D = np.full((places, B.shape[1]), np.nan)
    tol = np.zeros_like(D)
    for g, (a, b) in enumerate(_spans(offsets, places)):
        x = _gather(A, rows, a, b)
        D[a:b] = x @ B[g].T
        tol[a:b] = _bound(np.abs(x) @ np.abs(B[g]).T, B.shape[2], D[a:b], kind)
    return D, tol


def gradients(dD, A, B, offsets, rows, kind, kind_b):
    """dA, dB and their bounds; kind, kind_b: their types."""
    places = dD.shape[0]
    dA, dB = np.zeros((places, B.shape[2])), np.zeros(B.shape)
    ta, tb = np.zeros_like(dA), np.zeros_like(dB)
    for g, (a, b) in enumerate(_spans(offsets, places)):
        x, d = _gather(A, rows, a, b), dD[a:b]
        dA[a:b], dB[g] = d @ B[g], d.T @ x
        ta[a:b] = _bound(np.abs(d) @ np.abs(B[g]), B.shape[1], dA[a:b], kind)
        tb[g] = _bound(np.abs(d).T @ np.abs(x), b - a, dB[g], kind_b)
    return (dA, dB), (ta, tb)


def combine(X, slots, weights, kind):
    """out and its bound; slots and weights (tokens, top)."""
    t, top = slots.shape
    out, mag = np.zeros((t, X.shape[1])), np.zeros((t, X.shape[1]))
    for i in range(t):
        for j in range(top):
            if 0 <= slots[i, j] < X.shape[0]:
                out[i] += weights[i, j] * X[slots[i, j]]
                mag[i] += np.abs(weights[i, j] * X[slots[i, j]])
    return out, _bound(mag, top, out, kind)


def combine_gradients(dout, X, slots, rows, weights, kind):
    """dX, dw and their bounds."""
    t, top = slots.shape
    dX, dw, tx, tw = np.zeros(X.shape), np.zeros((t, top)), np.zeros(X.shape), np.zeros((t, top))
    for i, r in enumerate(rows):
        if not 0 <= r < t:
            continue
        js = [j for j in range(top) if slots[r, j] == i]
        w = sum(weights[r, j] for j in js)
        dX[i] = w * dout[r]
        tx[i] = _bound(sum(abs(weights[r, j]) for j in js) * np.abs(dout[r]), len(js), dX[i], kind)
        for j in js:
            dw[r, j] = dout[r] @ X[i]
            tw[r, j] = _bound(np.abs(dout[r]) @ np.abs(X[i]), X.shape[1], dw[r, j], "f32")
    return (dX, dw), (tx, tw)


def adapters(x, W, A, B, offsets, rows, scale, kind):
    """D (NaN in rows that no place leads to) and its bound.  The low-rank
    term's own factor is an fp32 sum, scaled and held in fp32; as an operand it
    may be off by 2^-38 of the row's largest besides."""
    places = x.shape[0] if rows is None else len(rows)
    r = np.arange(places) if rows is None else np.asarray(rows)
    K, R = W.shape[1], A.shape[1]
    D, tol = np.full((x.shape[0], W.shape[0]), np.nan), np.zeros((x.shape[0], W.shape[0]))
    group = np.full(places, -1)
    for g, (a, b) in enumerate(_spans(offsets, places)):
        group[a:b] = g
    for i in range(places):
        if not 0 <= r[i] < x.shape[0]:
            continue
        v, g = x[r[i]], group[i]
        want, mag = W @ v, np.abs(W) @ np.abs(v)
        err = 2 * (K + R + 16) * F32 * mag
        if g >= 0:
            h = scale[g] * (A[g] @ v)
            s = abs(scale[g])
            eh = 2 * (K + 8) * (F32 * s * (np.abs(A[g]) @ np.abs(v)) + (1 + s) * LOW) + \
                2 * F32 * np.abs(h) + 2.0 ** -38 * np.abs(h).max()
            want = want + B[g] @ h
            err = err + np.abs(B[g]) @ eh + 2 * (K + R + 16) * F32 * (np.abs(B[g]) @ np.abs(h))
        D[r[i]] = want
        tol[r[i]] = (1 + UNIT[kind]) * err + UNIT[kind] * np.abs(want) + TINY[kind] + \
            2 * (K + R) * LOW
    return D, tol
