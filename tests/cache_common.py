"""Shared helpers of the ragged and the shared-prefix decode tests.

Tolerances. bf16 P (half a step: 2^-8 of each weight) and bf16 O (2^-8 of the
result): |O - O_ref| <= 2^-8 (1 + 2^-6) O_abs + 2^-8 |O_ref|, O_abs the oracle's
output on |V|; the 2^-6 covers the fp32 parts below. A score is a sum of d
products in fp32, off by at most (d + 2) 2^-24 sum |q_d k_d| scale: E. LSE is off
by E, by 2^-22 of the exponentials and their sums' logarithm, and by fp32
roundings of its value: E + 2^-20 + 2^-22 |LSE|. A position's weight exp(s - LSE)
is off by E + (the same of LSE) of itself, and the sum it is added to rounds
g + 1 times: (2 E + 2^-19 + 2^-22 |LSE|) added + (g + 1) 2^-24 |W|.
"""

import numpy as np

import oracle
from causal_gqa_prefill_gb300 import workloads as W
from gpu_common import to_np


def make(B, C, n_q, n_kv, lens, seed=0, weights=True, junk=True):
    """Inputs of a step; with ``junk``, NaN and infinities behind every sequence."""
    import torch

    w = W.custom(B, 1, n_q, n_kv, 128, Lk=C)
    q, k, v = W.make_inputs(w, "cuda", seed=seed)
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if junk:
        behind = torch.arange(C, device="cuda")[None] >= lens[:, None]
        for x, bad in ((k, float("nan")), (v, float("inf"))):
            x[behind] = bad
    acc = None
    if weights:
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        acc = torch.rand(B, n_kv, C, generator=g, device="cuda")
        if junk:
            acc[behind[:, None].expand(-1, n_kv, -1)] = float("nan")
    return q, k, v, lens, acc


def check(q, k, v, lens, before, o, lse, after, scale=None, what="", prefix=None):
    """A step's outputs, and the weights before and after it (None: without)."""
    B, C, n_kv, d = k.shape
    g = q.shape[2] // n_kv
    o_r, lse_r, added, o_abs, s_abs = oracle.cache.decode_rows(
        to_np(q), to_np(k), to_np(v), lens.cpu().numpy(), scale=scale,
        **({} if prefix is None else {"prefix_k": to_np(prefix[0]), "prefix_v": to_np(prefix[1])}))
    o, lse = to_np(o), lse.cpu().numpy().astype(np.float64)
    bound = 2.0 ** -8 * ((1 + 2.0 ** -6) * o_abs + np.abs(o_r))
    assert (np.abs(o - o_r) <= bound).all(), (what, (np.abs(o - o_r) - bound).max())
    live = np.isfinite(lse_r)
    assert (lse[~live] == -np.inf).all(), what
    E = (d + 2) * 2.0 ** -24 * s_abs
    size = np.where(live, np.abs(lse_r), 0.0)
    bound = E + 2.0 ** -20 + 2.0 ** -22 * size
    off = np.abs(lse[live] - lse_r[live]) - bound[live]
    assert (off <= 0).all(), (what, off.max())
    if after is None:
        return
    rel = (2 * E + 2.0 ** -19 + 2.0 ** -22 * size)[..., 0].reshape(B, n_kv, g).max(2)[..., None]
    seen = np.arange(C)[None] < np.clip(lens.cpu().numpy(), 0, C)[:, None]
    seen = np.broadcast_to(seen[:, None], added.shape)
    ref = before.cpu().numpy().astype(np.float64) + added
    bound = rel * added + (g + 1) * 2.0 ** -24 * np.abs(ref)
    err = np.abs(after.cpu().numpy().astype(np.float64) - ref)
    assert (err[seen] <= bound[seen]).all(), (what, (err - bound)[seen].max())
    # entries behind a sequence keep their bits
    same = before.cpu().numpy().view(np.int32) == after.cpu().numpy().view(np.int32)
    assert same[~seen].all(), what
