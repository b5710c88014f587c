"""fp64 reference of the cache operators: key weights, ragged decode, eviction,
decode behind a shared prefix.

TEST INFRASTRUCTURE ONLY, like the rest of this package: written from the
definitions, one row or one head at a time, no tiling and no online softmax.

    kv(h) = h // g,  g = n_q / n_kv
    key weights   W[b,u,j] = sum over h in group u, rows i that see key j, of
                  exp(s_ihj - LSE_ih)
    ragged decode one row per sequence over its first lens[b] keys; a sequence
                  without keys gives o = 0 and lse = -inf
    eviction      the last R positions, and the N - R of largest weight before
                  them (ties to the lowest position, NaN lowest), in order
    shared prefix one row per sequence over P shared keys and its own lens[b]
"""

from __future__ import annotations

import numpy as np


def _softmax_row(s, v):
    """(o, lse, p) of one row of scores s [n] and values v [n, d]."""
    if len(s) == 0:
        return np.zeros(v.shape[1]), -np.inf, s
    m = s.max()
    e = np.exp(s - m)
    total = e.sum()
    return (e @ v) / total, m + np.log(total), e / total


def key_weights(q, k, lse, *, causal=True, scale=None):
    """W [B, n_kv, Lk] from q [B, Lq, n_q, d], k [B, Lk, n_kv, d], lse [B, n_q, Lq].

    Row i sits at position i + Lk - Lq. A row whose lse is -inf has no keys and
    adds nothing, whatever its q holds."""
    B, Lq, n_q, d = q.shape
    Lk, n_kv = k.shape[1], k.shape[2]
    g = n_q // n_kv
    scale = d ** -0.5 if scale is None else scale
    w = np.zeros((B, n_kv, Lk))
    for b in range(B):
        for h in range(n_q):
            s = scale * (q[b, :, h] @ k[b, :, h // g].T)
            live = lse[b, h] != -np.inf
            # (a choice, not a product with 0: its scores may be NaN or infinite)
            p = np.where(live[:, None], np.exp(s - np.where(live, lse[b, h], 0.0)[:, None]), 0.0)
            if causal:
                p = np.where(np.arange(Lk)[None] <= np.arange(Lq)[:, None] + Lk - Lq, p, 0.0)
            w[b, h // g] += p.sum(0)
    return w


def decode_rows(q, k, v, lens, *, prefix_k=None, prefix_v=None, scale=None):
    """(o [B, 1, n_q, d], lse [B, n_q, 1], added [B, n_kv, C], o_abs, s_abs).

    ``added`` is what the step adds to the weights of the sequence's own
    positions; o_abs [like o] the output with |v| for v, s_abs [B, n_q, 1] the
    largest scale * sum_d |q_d k_jd| of the row: what a rounding of a weight, or
    of a product in a score, is measured by."""
    B, _, n_q, d = q.shape
    C, n_kv = k.shape[1], k.shape[2]
    g = n_q // n_kv
    scale = d ** -0.5 if scale is None else scale
    o, o_abs = np.zeros((B, 1, n_q, d)), np.zeros((B, 1, n_q, d))
    lse, s_abs = np.full((B, n_q, 1), -np.inf), np.zeros((B, n_q, 1))
    added = np.zeros((B, n_kv, C))
    for b in range(B):
        n = min(max(int(lens[b]), 0), C)
        for h in range(n_q):
            u = h // g
            ks, vs = k[b, :n, u], v[b, :n, u]
            if prefix_k is not None:
                ks = np.concatenate([prefix_k[0, :, u], ks])
                vs = np.concatenate([prefix_v[0, :, u], vs])
            row, top, p = _softmax_row(scale * (ks @ q[b, 0, h]), vs)
            o[b, 0, h], lse[b, h, 0] = row, top
            if len(p):
                o_abs[b, 0, h] = p @ np.abs(vs)
                s_abs[b, h, 0] = abs(scale) * (np.abs(ks) @ np.abs(q[b, 0, h])).max()
                added[b, u, :n] += p[len(p) - n:]
    return o, lse, added, o_abs, s_abs


def evicted_index(weights, lens, budget, recent):
    """(index [B, n_kv, budget], -1 past the end, new lens [B])."""
    B, n_kv, C = weights.shape
    index = np.full((B, n_kv, budget), -1, dtype=np.int32)
    new = np.zeros(B, dtype=np.int32)
    for b in range(B):
        n = min(max(int(lens[b]), 0), C)
        new[b] = min(n, budget)
        for u in range(n_kv):
            if n <= budget:
                keep = np.arange(n)
            else:
                old = n - recent
                w = weights[b, u, :old].astype(np.float64)
                nan = np.isnan(w)
                order = np.lexsort((np.arange(old), -np.where(nan, 0.0, w), nan))
                keep = np.concatenate([np.sort(order[:budget - recent]), np.arange(old, n)])
            index[b, u, :len(keep)] = keep
    return index, new
