"""float64 attention over packed sequences, its gradients, and the error
bounds of a kernel that keeps sums in fp32 and rounds weights, score
gradients and results once to a 16-bit type.

Definition, per sequence with lq query tokens and lk keys, query head h of kv
head g = h // (heads // kv heads):

    s_tj = scale * q_t . k_j      j visible: j <= t + lk - lq (causal) or all
    lse_t = log sum_j exp(s_tj),  p = exp(s - lse),  out_t = sum_j p_tj v_j
    dV_j = sum_t p_tj dO_t        dS = p (dO V^T - rowsum(dO out))
    dQ = scale dS K               dK = scale dS^T Q

Rows without a visible key: out 0, lse -inf.  Arrays are float64; 16-bit
values are exact in them.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

# half a step of the type, relative; half of its smallest step, absolute
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}
F32 = 2.0 ** -24
NORMAL = 2.0 ** -126     # fp32's least normal: an exponential below it is 0


@dataclass
class Head:
    """One sequence and head: the pieces the bounds need."""
    s: np.ndarray       # scores, -inf where hidden
    p: np.ndarray
    lse: np.ndarray
    out: np.ndarray


def visible(lq: int, lk: int, causal: bool) -> np.ndarray:
    if not causal:
        return np.ones((lq, lk), bool)
    return np.arange(lk)[None, :] <= np.arange(lq)[:, None] + (lk - lq)


def one_head(q, k, v, scale: float, seen: np.ndarray) -> Head:
    s = np.where(seen, scale * (q @ k.T), -np.inf)
    top = s.max(axis=1, initial=-np.inf)
    safe = np.where(np.isneginf(top), 0.0, top)
    w = np.exp(s - safe[:, None])
    total = w.sum(axis=1)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, safe + np.log(total), -np.inf)
    p = w / np.where(total > 0, total, 1.0)[:, None]
    return Head(s, p, lse, p @ v)


def _eta(q, k, seen, scale, dim):
    """Error of a score, at most, in units of its exponent: the fp32 sum of
    the products (each addition off by half a step of the running sum, the
    instruction's own additions not better than truncation: twice that), the
    product with scale log2 e and the exponential's own error."""
    mag = scale * (np.abs(q) @ np.abs(k).T)
    mag = np.where(seen, mag, 0.0).max(initial=0.0)
    return 2 * (dim + 8) * F32 * mag + 8 * F32


def attention(q, k, v, seq_q, seq_k, causal, scale, kind):
    """out, lse and their error bounds for q (tokens, heads, dim), k and v
    (keys, kv heads, dim); tokens of no sequence are NaN."""
    t, h, d = q.shape
    g = h // k.shape[1]
    out, lse = np.full(q.shape, np.nan), np.full((t, h), np.nan)
    tol, tol_lse = np.zeros(q.shape), np.zeros((t, h))
    u, tiny = UNIT[kind], TINY[kind]
    for a, b, x, y in zip(seq_q[:-1], seq_q[1:], seq_k[:-1], seq_k[1:]):
        seen = visible(b - a, y - x, causal)
        for i in range(h):
            qi, ki, vi = q[a:b, i], k[x:y, i // g], v[x:y, i // g]
            r = one_head(qi, ki, vi, scale, seen)
            out[a:b, i], lse[a:b, i] = r.out, r.lse
            n = y - x
            eta = _eta(qi, ki, seen, scale, d)
            mag = r.p @ np.abs(vi)
            # weights: one rounding, their scores' error, the fp32 sums of
            # numerator and denominator; the quotient; one rounding
            tol[a:b, i] = mag * (u + 2 * eta + 4 * (n + 8) * F32) + \
                tiny * 256 * np.abs(vi).sum(axis=0, initial=0.0) + u * np.abs(r.out) + tiny
            fin = np.where(np.isfinite(r.lse), np.abs(r.lse), 0.0)
            tol_lse[a:b, i] = eta + 2 * (n + 8) * F32 + 4 * F32 * (fin + 16)
    return out, lse, tol, tol_lse


def gradients(dout, q, k, v, out, lse, seq_q, seq_k, causal, scale, kind):
    """dq, dk, dv for the given out and lse (inputs, as the kernel takes
    them), and their error bounds."""
    h, d = q.shape[1:]
    g = h // k.shape[1]
    u, tiny = UNIT[kind], TINY[kind]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    tq, tk, tv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for a, b, x, y in zip(seq_q[:-1], seq_q[1:], seq_k[:-1], seq_k[1:]):
        seen = visible(b - a, y - x, causal)
        for i in range(h):
            j = i // g
            qi, ki, vi, do, o = q[a:b, i], k[x:y, j], v[x:y, j], dout[a:b, i], out[a:b, i]
            z = lse[a:b, i]
            fin = np.isfinite(z)
            s = scale * (qi @ ki.T)
            p = np.where(seen & fin[:, None], np.exp(s - np.where(fin, z, 0.0)[:, None]), 0.0)
            dp = do @ vi.T
            delta = (do * o).sum(axis=1)
            ds = p * (dp - delta[:, None])
            eta = _eta(qi, ki, seen, scale, d) + 4 * F32 * (np.abs(z[fin]).max(initial=0.0) + 16)
            dv[x:y, j] += p.T @ do
            dq[a:b, i] = scale * (ds @ ki)
            dk[x:y, j] += scale * (ds.T @ qi)
            # a score gradient: its weight's error, the fp32 sums of dP and
            # delta, one rounding.  A weight below 2^-126 is formed as 0: off by
            # less than that, its score gradient by that times |dP - delta|
            # (for a key that no row gives more this is all of its gradient)
            sums = 2 * (d + 8) * F32 * (np.abs(do) @ np.abs(vi).T +
                                        (np.abs(do) * np.abs(o)).sum(axis=1)[:, None])
            eds = np.abs(ds) * (u + 2 * eta + 4 * F32) + p * sums + \
                np.where(seen, tiny + NORMAL * np.abs(dp - delta[:, None]), 0.0)
            ep = p * (u + 2 * eta) + np.where(seen, tiny + NORMAL, 0.0)
            n, m = y - x, (b - a) * g
            tq[a:b, i] = scale * ((eds + 2 * (n + 8) * F32 * np.abs(ds)) @ np.abs(ki))
            tk[x:y, j] += scale * ((eds + 2 * (m + 8) * F32 * np.abs(ds)).T @ np.abs(qi))
            tv[x:y, j] += (ep + 2 * (m + 8) * F32 * p).T @ np.abs(do)
    tq += u * np.abs(dq) + tiny + 2 * F32 * np.abs(dq)
    tk += u * np.abs(dk) + tiny + 2 * F32 * np.abs(dk)
    tv += u * np.abs(dv) + tiny + 2 * F32 * np.abs(dv)
    return (dq, dk, dv), (tq, tk, tv)


def prefix_attention(q, prefix_k, prefix_v, k, v, lengths, scale, kind):
    """out, lse and bounds for q (batch, tokens, heads, dim), the prefix
    (keys, kv heads, dim) and caches (batch, capacity, kv heads, dim): token t
    of `tokens` sees the prefix and the first lengths[b] - tokens + t + 1 keys
    of cache b."""
    b, t, h, d = q.shape
    g = h // prefix_k.shape[1]
    out, lse = np.zeros(q.shape), np.zeros((b, t, h))
    tol, tol_lse = np.zeros(q.shape), np.zeros((b, t, h))
    u, tiny = UNIT[kind], TINY[kind]
    n0 = prefix_k.shape[0]
    for i in range(b):
        n = min(max(int(lengths[i]), 0), k.shape[1])
        own = np.arange(n)[None, :] <= np.arange(t)[:, None] + (n - t)
        seen = np.concatenate([np.ones((t, n0), bool), own], axis=1)
        for x in range(h):
            ki = np.concatenate([prefix_k[:, x // g], k[i, :n, x // g]])
            vi = np.concatenate([prefix_v[:, x // g], v[i, :n, x // g]])
            r = one_head(q[i, :, x], ki, vi, scale, seen)
            out[i, :, x], lse[i, :, x] = r.out, r.lse
            eta = _eta(q[i, :, x], ki, seen, scale, d)
            total = n0 + n
            tol[i, :, x] = (r.p @ np.abs(vi)) * (u + 3 * eta + 4 * (total + 8) * F32) + \
                tiny * 256 * np.abs(vi).sum(axis=0, initial=0.0) + u * np.abs(r.out) + tiny
            fin = np.where(np.isfinite(r.lse), np.abs(r.lse), 0.0)
            tol_lse[i, :, x] = eta + 2 * (total + 8) * F32 + 4 * F32 * (fin + 16)
    return out, lse, tol, tol_lse
