"""Key weights where the ranges of steps that the CTAs get matter: against the fp64
oracle, with the ranges replayed here from their definition, so that each case says
which of the kernel's paths it takes.

A step is 128 // g query positions of one group against 256 keys; the steps of all
(sequence, K/V head, 256 keys) in order are cut into equal ranges, one per CTA.

Tolerance. A row's weight exp(s - LSE) is off by the score's fp32 error, at most
(d + 2) 2^-24 scale sum |q_d k_d|, by the roundings of c s - lse2 in the exponent
(its operands and its result: 2^-22 (|s| + |LSE|) covers their half steps and the
factor log2 e) and by 2^-22 of the exponential. A sum adds a step's weight to that of
the steps before it in the range (at most all that one range holds of a unit), folds
32 lanes (5 additions) and four warps (3) and adds the ranges that a unit is cut into:
2^-24 each, of positive terms, so the relative bound carries over.
"""

import numpy as np
import pytest

import oracle
from causal_gqa_prefill_gb300 import ATTN_OK, attn_device_check, attn_key_weights, attn_prefill
from causal_gqa_prefill_gb300 import workloads as W
from gpu_common import to_np

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CTAS, KEYS, ROWS = 152, 256, 128
RING = {128: 3, 64: 6}        # steps whose query rows fit shared memory at once


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def ranges(B, Lq, Lk, n_q, n_kv, causal):
    """[[(head, unit, step), ...] per CTA], and the steps that each unit has."""
    nr = ROWS // (n_q // n_kv)
    steps, off = -(-Lq // nr), Lk - Lq
    units = [range(max(t * KEYS - off, 0) // nr if causal else 0, steps)
             for t in range(-(-Lk // KEYS))]
    every = [(h, t, s) for h in range(B * n_kv) for t, u in enumerate(units) for s in u]
    G = min(CTAS, len(every))
    return [every[c * len(every) // G:(c + 1) * len(every) // G] for c in range(G)], units


def additions(cuts):
    """The most additions that lead to one weight."""
    held, cut = {}, {}
    for c, r in enumerate(cuts):
        for h, t, _ in r:
            held[c, h, t] = held.get((c, h, t), 0) + 1
    for c, h, t in held:
        cut[h, t] = cut.get((h, t), 0) + 1
    return max(held.values()) + 5 + 3 + max(cut.values())


def inputs(B, Lq, Lk, n_q, n_kv, d, causal, seed):
    w = W.custom(B, Lq, n_q, n_kv, d, causal=causal, Lk=Lk)
    q, k, v = W.make_inputs(w, "cuda", seed=seed)
    _, lse = attn_prefill(q, k, v, causal=causal)
    return q, k, lse


def check(q, k, lse, got, causal, cuts, before=None):
    qn, kn, ln = to_np(q), to_np(k), lse.cpu().numpy().astype(np.float64)
    d, scale = q.shape[3], q.shape[3] ** -0.5
    ref = oracle.cache.key_weights(qn, kn, ln, causal=causal)
    live = np.isfinite(ln)
    size = scale * np.linalg.norm(qn, axis=3).max() * np.linalg.norm(kn, axis=3).max()
    rel = ((d + 2) * 2.0 ** -24 * size + 2.0 ** -22 * (size + np.abs(ln[live]).max()) + 2.0 ** -22
           + additions(cuts) * 2.0 ** -24)
    bound = rel * ref
    if before is not None:
        ref = ref + before.cpu().numpy().astype(np.float64)
        bound = bound + 2.0 ** -24 * np.abs(ref)
    err = np.abs(got.cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound).all(), (err / np.maximum(bound, 1e-300)).max()


# B, Lq, Lk, n_q, n_kv, d: all steps of a head fit the ring, and a CTA has several heads
STAY = [
    (8, 60, 1500, 48, 8, 128),      # 3 steps, g = 6: 126 of 128 rows
    (8, 60, 1500, 48, 8, 64),
    (8, 60, 1300, 96, 8, 64),       # 6 steps, g = 12; hidden ones in the last unit
    (20, 90, 600, 32, 8, 128),      # 3 steps, g = 4, the last one mostly rows of the one before
    (30, 3, 700, 256, 2, 128),      # 3 steps of one row, g = 128
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", STAY, ids=lambda c: "B%d_%dx%d_q%d_kv%d_d%d" % c)
def test_query_rows_that_stay(case, causal):
    """Query rows kept from unit to unit and replaced where the head changes, also in
    CTAs whose range leaves some of a head's steps out, at its start and at its end."""
    B, Lq, Lk, n_q, n_kv, d = case
    cuts, units = ranges(B, Lq, Lk, n_q, n_kv, causal)
    steps = units[0].stop
    assert steps <= RING[d] and Lq * n_q // n_kv > 256
    kept = left_out_first = left_out_last = 0
    for r in cuts:
        heads = list(dict.fromkeys(h for h, _, _ in r))
        used = [{s for h, _, s in r if h == head} for head in heads]
        kept += any(len({t for h, t, _ in r if h == head}) > 1 for head in heads)
        left_out_first += len(heads) > 1 and len(used[0]) < steps
        left_out_last += len(used[-1]) < steps
    assert kept and left_out_first and left_out_last
    q, k, lse = inputs(*case, causal, seed=sum(case))
    first = attn_key_weights(q, k, lse, causal=causal)
    assert attn_device_check() == ATTN_OK
    check(q, k, lse, first, causal, cuts)
    for _ in range(20):                             # back to back: the same bits
        again = attn_key_weights(q, k, lse, causal=causal)
    assert torch.equal(again, first)
    before = torch.rand(first.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    got = before.clone()
    attn_key_weights(q, k, lse, causal=causal, weights=got, accumulate=True)
    check(q, k, lse, got, causal, cuts, before=before)


# whole units of several steps, and several units a CTA, beside units that are cut
WHOLE = [
    # B, Lq, Lk, n_q, n_kv, d
    (40, 513, 513, 16, 4, 128),     # 17 steps a unit, g = 4
    (40, 300, 900, 16, 4, 64),      # a chunk
    (120, 257, 400, 12, 2, 64),     # g = 6
    (60, 200, 300, 40, 5, 128),     # g = 8
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", WHOLE, ids=lambda c: "B%d_%dx%d_q%d_kv%d_d%d" % c)
def test_whole_units_of_several_steps(case, causal):
    """Units that one CTA sums alone, step after step, written and added to."""
    B, Lq, Lk, n_q, n_kv, d = case
    cuts, units = ranges(B, Lq, Lk, n_q, n_kv, causal)
    assert units[0].stop > RING[d]                  # the rows pass through the ring
    alone = sum(len(u) > 1 and [s for h2, t2, s in r if (h2, t2) == (h, t)] == list(u)
                for r in cuts for h, t in dict.fromkeys((h, t) for h, t, _ in r)
                for u in [units[t]])
    assert alone > CTAS and len(units) * B * n_kv > alone
    q, k, lse = inputs(*case, causal, seed=sum(case))
    first = attn_key_weights(q, k, lse, causal=causal)
    assert attn_device_check() == ATTN_OK
    check(q, k, lse, first, causal, cuts)
    before = torch.rand(first.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    got = before.clone()
    attn_key_weights(q, k, lse, causal=causal, weights=got, accumulate=True)
    check(q, k, lse, got, causal, cuts, before=before)


@pytest.mark.parametrize("n_q", [8, 32])
def test_many_steps_in_one_sum(n_q):
    """Few keys and many rows: hundreds of steps of one unit in one CTA."""
    case = (1, 16384, 16384, n_q, 2, 64)
    cuts, _ = ranges(*case[:5], True)
    assert max(len(r) for r in cuts) > 200
    q, k, lse = inputs(*case, True, seed=n_q)
    got = attn_key_weights(q, k, lse).double()
    assert attn_device_check() == ATTN_OK
    keys = torch.tensor([0, 1, 255, 256, 5000, 8191, 16000, 16383], device="cuda")
    size = 64 ** -0.5 * (q.float().norm(dim=3).max() * k.float().norm(dim=3).max()).item()
    rel = (66 * 2.0 ** -24 * size + 2.0 ** -22 * (size + lse.abs().max().item()) + 2.0 ** -22
           + additions(cuts) * 2.0 ** -24)
    g, rows = n_q // 2, torch.arange(16384, device="cuda")
    for u in range(2):
        ref = torch.zeros(len(keys), dtype=torch.float64, device="cuda")
        for h in range(g * u, g * u + g):
            s = q[0, :, h].double() @ k[0, keys, u].double().T * 64 ** -0.5
            p = torch.exp(s - lse[0, h].double()[:, None])
            ref += torch.where(keys[None] <= rows[:, None], p, 0.0).sum(0)
        assert ((got[0, u, keys] - ref).abs() <= rel * ref).all()
