"""4-bit decode where every warp has a run of many chunks of 16 positions: full steps, a
ring that is filled again and again, heads that end inside a run, runs that go from a
head's sinks to its window and over several heads, both kernels (groups of up to 8
query heads and of more).

Tolerance: test_gpu_cache4's, and what sums that go on for long add. Of a head a warp
adds n chunks one after another, n at most its run's length: per chunk one product to
an output and two weights and two weights times mid to its lane's sums, each of them off
by a step of fp32 at most, 2^-23, and every two chunks perhaps one rescaling, 2^-24 of
each. A head's parts in m warps are added one after another too. So outputs and sums are
off by (n + m) (2^-22 + 2^-25) < (n + m) 2^-21.8 of what they add up: sum p (|V - mid| +
|mid|) and the sum of the weights. |mid| <= |lo| + |V| (mid is lo, the group's largest
value or, between them, half a scale at most), so that is at most 3 sum p (|lo| + |V|):
    (n + m) 2^-20 (sum p (|lo| + |V|) + |O|) on O,  (n + m) 2^-21 on LSE.
"""

import numpy as np
import pytest

from causal_gqa_prefill_gb300 import ATTN_OK, attn_decode4, attn_device_check, attn_pack4
from causal_gqa_prefill_gb300 import workloads as W
from gpu_common import to_np
from oracle import cache4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def seen(n, window, sinks):
    first = max(0, n - window) if window else 0
    return min(sinks, first), first


def chunks(n, window, sinks):
    sunk, first = seen(n, window, sinks)
    return -(-sunk // 16) + -(-(n - first) // 16)


def make(B, C, n_q, n_kv, lens, window, sinks, seed):
    """A step's inputs; scales and lowest values are NaN wherever no token looks."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    caches = [torch.zeros(B, n_kv, C, 80, dtype=torch.uint8, device="cuda") for _ in range(2)]
    k, v = (torch.randn(B, C, n_kv, 128, generator=gen, device="cuda") for _ in range(2))
    k[..., 5::32] *= 8
    attn_pack4(k.to(torch.bfloat16), v.to(torch.bfloat16), *caches)
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    at, end = torch.arange(C, device="cuda")[None], lens.long()[:, None]
    hidden = at >= end
    if window:
        hidden |= (at < end - window) & (at >= sinks)
    for c in caches:
        c.transpose(1, 2)[hidden] = 255
    q = W.make_inputs(W.custom(B, 1, n_q, n_kv, 128, Lk=4), "cuda", seed=seed)[0]
    return q, *caches, lens


def values(rows):
    """(what rows stand for, lo, scale), each [n, 128]."""
    val, lo = cache4.unpack(rows)
    word = rows[:, 64:].reshape(-1, 4, 4).astype(np.uint32)
    return val, lo, np.repeat(cache4.bf16_value(word[..., 0] | word[..., 1] << 8), 32, axis=1)


def check(q, k4, v4, lens, o, lse, window, sinks):
    q, o, lse = to_np(q), to_np(o), lse.cpu().numpy().astype(np.float64)
    k4, v4 = k4.cpu().numpy(), v4.cpu().numpy()
    n_kv, n_q = k4.shape[1], q.shape[2]
    g, lens = n_q // n_kv, lens.tolist()
    warps = 152 * (12 if g <= 8 else 8)
    run = -(-sum(chunks(n, window, sinks) for n in lens) * n_kv // warps)
    for b, n in enumerate(lens):
        if n == 0:
            assert not o[b].any() and (lse[b] == -np.inf).all()
            continue
        sunk, first = seen(n, window, sinks)
        at = [*range(sunk), *range(first, n)]
        own = chunks(n, window, sinks)
        adds = min(run, own) + -(-own // max(1, run - 1)) + 2
        for u in range(n_kv):
            (K, klo, kstep), (V, vlo, vstep) = (values(c[b, u, at]) for c in (k4, v4))
            Q, heads = q[b, 0, u * g:u * g + g], slice(u * g, u * g + g)
            s = 128 ** -0.5 * (Q @ K.T)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(1, keepdims=True)
            p /= total
            ref, ref_lse = p @ V, (m + np.log(total))[:, 0]
            E = 2.0 ** -20 * 128 ** -0.5 * (np.abs(Q) @ (47 * kstep + np.abs(klo)).T).max(1)
            off = np.abs(lse[b, heads, 0] - ref_lse)
            assert (off <= E + 2.0 ** -20 + adds * 2.0 ** -21 + 2.0 ** -22 * np.abs(ref_lse)).all()
            with np.errstate(divide="ignore", invalid="ignore"):
                code = np.where(vstep > 0, -vlo / vstep, 0.0)
            near = np.abs(code - np.floor(code) - 0.5) < 2.0 ** -16
            mid = vlo + vstep * np.clip(np.rint(code), 0, 15)
            A = p @ (np.abs(V - mid) + near * vstep)
            bound = 2.0 ** -8 * ((1 + 2.0 ** -6) * A + np.abs(ref)) + (
                2 * E[:, None] + (1 + adds) * 2.0 ** -20) * (
                    p @ (np.abs(vlo) + np.abs(V)) + np.abs(ref))
            err = np.abs(o[b, 0, heads] - ref)
            assert (err <= bound).all(), (b, u, (err - bound).max())


def spread(B, C, zero=()):
    """Lengths over the whole range, in no order."""
    return [0 if b in zero else 1 + (b * 7919) % C for b in range(B)]


RUNS = [
    # B, C, n_q, n_kv, lens, window, sinks, chunks a warp at least
    (1, 20000, 72, 8, [19999], None, 0, 8),                  # g = 9
    (2, 10003, 48, 4, [10003, 9990], None, 0, 4),            # g = 12
    (1, 20000, 128, 8, [20000], None, 0, 8),                 # g = 16
    (40, 2000, 96, 6, spread(40, 2000, (7, 39)), None, 0, 10),       # heads end inside runs, g = 16
    (90, 1000, 36, 3, spread(90, 1000, (0, 44)), None, 0, 6),        # g = 12
    (1, 150000, 16, 2, [149995], None, 0, 10),               # g = 8
    (24, 6000, 20, 5, spread(24, 6000, (3,)), None, 0, 10),  # g = 4
    (200, 300, 32, 8, spread(200, 300, (50, 199)), 100, 20, 5),      # sinks, window, several heads
    (600, 150, 32, 8, spread(600, 150, (0, 1, 2, 300)), 24, 5, 5),   # three heads a run
    (700, 60, 16, 8, spread(700, 60, (9, 10)), 1, 1, 4),     # two chunks of one position a head
    (200, 300, 80, 8, spread(200, 300, (50, 199)), 100, 20, 8),      # the same, g = 10
    (500, 150, 96, 8, spread(500, 150, (0, 1, 2, 300)), 24, 5, 6),   # g = 12
    (300, 500, 64, 4, spread(300, 500, (5,)), 200, 33, 8),   # g = 16
    (64, 4000, 32, 4, spread(64, 4000, (63,)), 1024, 4, 6),  # g = 8
]


@pytest.mark.parametrize("case", RUNS, ids=lambda c: "B%d_C%d_q%d_kv%d_W%s_S%d" % (c[:4] + c[5:7]))
def test_long_runs(case):
    B, C, n_q, n_kv, lens, window, sinks, least = case
    per = sum(chunks(n, window, sinks) for n in lens) * n_kv / (152 * (12 if n_q // n_kv <= 8 else 8))
    assert per >= least
    q, k4, v4, lens = make(B, C, n_q, n_kv, lens, window, sinks, seed=B + C)
    o, lse = attn_decode4(q, k4, v4, lens, window=window, sinks=sinks)
    assert attn_device_check() == ATTN_OK
    check(q, k4, v4, lens, o, lse, window, sinks)
    again = attn_decode4(q, k4, v4, lens, window=window, sinks=sinks)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
