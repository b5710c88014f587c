"""fp64 reference of attention behind a sliding window with sinks.

TEST INFRASTRUCTURE ONLY, like the rest of this package: written from the
definition, one head at a time, no tiling and no online softmax.

    row i of Lq sits at position p = i + Lk - Lq and sees the keys
    j <= p  with  j > p - window  or  j < sinks
"""

from __future__ import annotations

import numpy as np


def seen(Lq, Lk, window, sinks):
    """bool [Lq, Lk]: which keys each row sees."""
    p = np.arange(Lq)[:, None] + Lk - Lq
    j = np.arange(Lk)[None]
    return (j <= p) & ((j > p - window) | (j < sinks))


def _scores(q, k, scale):
    """scale * q k^T, and scale * |q| |k|^T: what a rounding in a score is measured by."""
    return scale * (q @ k.T), abs(scale) * (np.abs(q) @ np.abs(k).T)


def attention(q, k, v, window, sinks, scale=None):
    """(o, lse, o_abs, s_abs) of q [B, Lq, n_q, d], k, v [B, Lk, n_kv, d].

    o_abs [like o] is the output with |v| for v, s_abs [like lse] the largest
    scale * sum_d |q_d k_jd| of the row. Keys that a row does not see may hold
    anything."""
    B, Lq, n_q, d = q.shape
    Lk, n_kv = k.shape[1], k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    see = seen(Lq, Lk, window, sinks)
    any_row = see.any(0)
    o, o_abs = np.zeros(q.shape), np.zeros(q.shape)
    lse, s_abs = np.zeros((B, n_q, Lq)), np.zeros((B, n_q, Lq))
    for b in range(B):
        for h in range(n_q):
            u = h // (n_q // n_kv)
            kk = np.where(any_row[:, None], k[b, :, u], 0.0)
            vv = np.where(any_row[:, None], v[b, :, u], 0.0)
            s, sa = _scores(q[b, :, h], kk, scale)
            s = np.where(see, s, -np.inf)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            total = e.sum(1, keepdims=True)
            o[b, :, h] = (e @ vv) / total
            o_abs[b, :, h] = (e @ np.abs(vv)) / total
            lse[b, h] = (m + np.log(total))[:, 0]
            s_abs[b, h] = np.where(see, sa, 0.0).max(1)
    return o, lse, o_abs, s_abs


def backward(q, k, v, o, lse, dout, window, sinks, scale=None):
    """Gradients (dq, dk, dv) from the forward's o and lse, and for each the sum of
    the magnitudes that roundings of P and dS are measured by (see the tests)."""
    B, L, n_q, d = q.shape
    n_kv = k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    see = seen(L, L, window, sinks)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)
    eq, ek, ev = np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)
    for b in range(B):
        for h in range(n_q):
            u = h // (n_q // n_kv)
            Q, K, V, G, O = q[b, :, h], k[b, :, u], v[b, :, u], dout[b, :, h], o[b, :, h]
            s, _ = _scores(Q, K, scale)
            p = np.where(see, np.exp(np.where(see, s, 0.0) - lse[b, h][:, None]), 0.0)
            ds = p * (G @ V.T - (G * O).sum(1, keepdims=True))
            dq[b, :, h] = scale * (ds @ K)
            dk[b, :, u] += scale * (ds.T @ Q)
            dv[b, :, u] += p.T @ G
            # bf16 dS: half a step, 2^-8, and 2^-12 = 2^-8 2^-4 for what fp32 does to P (its
            # score's error, 2^-13 for scores of up to 16) and to the sum over rows and heads
            # (up to 2^14 terms in runs of 16: 2^-13); the fp32 sums dP and D are off by
            # (d + 2) 2^-24 of their magnitudes each
            size = np.abs(G) @ np.abs(V).T + (np.abs(G) * np.abs(O)).sum(1, keepdims=True)
            e = 2.0 ** -8 * (1 + 2.0 ** -4) * np.abs(ds) + p * (d + 2) * 2.0 ** -24 * size
            eq[b, :, h] = abs(scale) * (e @ np.abs(K))
            ek[b, :, u] += abs(scale) * (e.T @ np.abs(Q))
            ev[b, :, u] += 2.0 ** -8 * (1 + 2.0 ** -4) * (p.T @ np.abs(G))
    return (dq, dk, dv), (eq, ek, ev)


def decode_rows(q, k, v, lens, window, sinks, scale=None):
    """(o, lse, o_abs, s_abs) of one token per sequence: q [B, 1, n_q, d] at position
    lens[b] - 1 of k, v [B, C, n_kv, d]; a sequence without keys gives o = 0 and
    lse = -inf. window None: everything before lens[b]."""
    B, _, n_q, d = q.shape
    C = k.shape[1]
    o, o_abs = np.zeros(q.shape), np.zeros(q.shape)
    lse, s_abs = np.full((B, n_q, 1), -np.inf), np.zeros((B, n_q, 1))
    for b in range(B):
        n = int(min(max(lens[b], 0), C))
        if n:
            w, s = (n, 0) if window is None else (window, sinks)
            r = attention(q[b:b + 1], k[b:b + 1, :n], v[b:b + 1, :n], w, s, scale)
            o[b], lse[b], o_abs[b], s_abs[b] = (x[0] for x in r)
    return o, lse, o_abs, s_abs
