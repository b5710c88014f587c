"""GPU parity of attention behind a sliding window with sinks: prefill, its
gradient and decode against the fp64 reference.

Tolerances. O and LSE as cache_common derives them: |O - O_ref| <= 2^-8 ((1 + 2^-6)
O_abs + |O_ref|), |LSE - LSE_ref| <= E + 2^-20 + 2^-22 |LSE_ref| with E =
(d + 2) 2^-24 S_abs. Gradients: the sums that oracle.window.backward returns
beside them, and half a bf16 step of the result, 2^-8 |G_ref|.
"""

import numpy as np
import pytest

from causal_gqa_prefill_gb300 import (ATTN_OK, attn_decode_ragged, attn_decode_window,
                                      attn_decode_window_workspace_bytes, attn_device_check,
                                      attn_prefill, attn_prefill_backward, attn_prefill_window,
                                      attn_prefill_window_backward,
                                      attn_prefill_window_bwd_workspace_bytes)
from causal_gqa_prefill_gb300 import workloads as W
from gpu_common import to_np
from oracle import window as ow

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def make(B, Lq, Lk, n_q, n_kv, d, seed=0):
    return W.make_inputs(W.custom(B, Lq, n_q, n_kv, d, Lk=Lk), "cuda", seed=seed)


def check_rows(o, lse, ref, d, what=""):
    o_r, lse_r, o_abs, s_abs = ref
    o, lse = to_np(o), lse.cpu().numpy().astype(np.float64)
    bound = 2.0 ** -8 * ((1 + 2.0 ** -6) * o_abs + np.abs(o_r))
    assert (np.abs(o - o_r) <= bound).all(), (what, (np.abs(o - o_r) - bound).max())
    live = np.isfinite(lse_r)
    assert (lse[~live] == -np.inf).all(), what
    bound = (d + 2) * 2.0 ** -24 * s_abs + 2.0 ** -20 + 2.0 ** -22 * np.where(live, np.abs(lse_r), 0)
    assert (np.abs(lse[live] - lse_r[live]) <= bound[live]).all(), what


# ------------------------------------------------------------------- prefill

FWD = [
    # B, Lq, Lk, n_q, n_kv, d, W, S
    (1, 1, 1, 1, 1, 64, 1, 0),
    (1, 1, 300, 4, 1, 128, 1, 0),                 # each row sees itself alone
    (2, 333, 333, 4, 1, 64, 100, 3),
    (1, 300, 300, 2, 2, 128, 128, 0),             # one head a group: neighbouring tiles in a unit
    (1, 520, 520, 3, 1, 128, 128, 5),             # an odd number of tiles, three heads a group
    (1, 520, 520, 3, 1, 128, 129, 130),           # more than a tile of sinks
    (1, 640, 640, 2, 1, 64, 127, 300),            # sinks that reach into the window's first tile
    (2, 400, 400, 6, 2, 128, 1, 1),
    (1, 257, 900, 8, 2, 128, 200, 64),            # a chunk
    (1, 100, 1000, 4, 4, 64, 37, 0),
    (1, 100, 1000, 4, 4, 64, 37, 905),            # all but a few positions are sinks
    (3, 5, 700, 10, 5, 128, 300, 1),
    (1, 256, 256, 4, 1, 128, 256, 0),             # nothing hidden
    (1, 256, 256, 4, 1, 128, 10 ** 12, 7),
    (1, 1500, 1500, 16, 1, 64, 400, 17),
    (1, 130, 4000, 2, 1, 128, 1000, 128),         # the sinks fill their tile
    (1, 700, 700, 1, 1, 128, 255, 256),
]


@pytest.mark.parametrize("case", FWD, ids=str)
def test_prefill(case):
    B, Lq, Lk, n_q, n_kv, d, win, sinks = case
    q, k, v = make(B, Lq, Lk, n_q, n_kv, d, seed=sum(case[:6]))
    o, lse = attn_prefill_window(q, k, v, win, sinks)
    assert attn_device_check() == ATTN_OK
    check_rows(o, lse, ow.attention(to_np(q), to_np(k), to_np(v), win, sinks), d, str(case))


def test_prefill_random_shapes():
    rng = np.random.default_rng(20)
    for n in range(60):
        n_kv = int(rng.choice([1, 2, 3]))
        n_q = n_kv * int(rng.choice([1, 2, 3, 4, 5, 8]))
        Lk = int(rng.integers(1, 900))
        Lq = Lk if n % 2 else int(rng.integers(1, Lk + 1))
        win, sinks = int(rng.integers(1, 500)), int(rng.choice([0, 1, 4, rng.integers(0, 400)]))
        B, d = int(rng.choice([1, 2])), int(rng.choice([64, 128]))
        q, k, v = make(B, Lq, Lk, n_q, n_kv, d, seed=n)
        o, lse = attn_prefill_window(q, k, v, win, sinks)
        check_rows(o, lse, ow.attention(to_np(q), to_np(k), to_np(v), win, sinks), d,
                   str((B, Lq, Lk, n_q, n_kv, d, win, sinks)))
    assert attn_device_check() == ATTN_OK


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5])
def test_prefill_other_scales(scale):
    q, k, v = make(1, 300, 400, 4, 2, 128, seed=5)
    o, lse = attn_prefill_window(q, k, v, 90, 6, scale=scale)
    check_rows(o, lse, ow.attention(to_np(q), to_np(k), to_np(v), 90, 6, scale=scale), 128)


def test_prefill_without_a_window_is_the_causal_one():
    q, k, v = make(2, 500, 700, 6, 2, 128, seed=6)
    o, lse = attn_prefill_window(q, k, v, 700)
    o2, lse2 = attn_prefill(q, k, v)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("win,sinks,Lq", [(100, 10, 64), (130, 0, 200), (40, 200, 3), (1, 1, 1),
                                          (127, 129, 129)])
def test_positions_that_no_row_sees_may_hold_anything(win, sinks, Lq):
    Lk = 900
    q, k, v = make(1, Lq, Lk, 4, 2, 128, seed=7)
    o, lse = attn_prefill_window(q, k, v, win, sinks)
    hidden = slice(sinks, max(sinks, Lk - Lq - win + 1))
    k[:, hidden], v[:, hidden] = float("nan"), float("inf")
    o2, lse2 = attn_prefill_window(q, k, v, win, sinks)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_rows(o, lse, ow.attention(to_np(q), to_np(k), to_np(v), win, sinks), 128)


def test_prefill_in_chunks_is_the_whole():
    q, k, v = make(1, 1000, 1000, 4, 2, 64, seed=8)
    o, lse = attn_prefill_window(q, k, v, 300, 9)
    at = 0
    for n in (1, 128, 371, 500):
        end = at + n
        part = [x.contiguous() for x in (q[:, at:end], k[:, :end], v[:, :end])]
        o2, lse2 = attn_prefill_window(*part, 300, 9)
        assert (o2.float() - o[:, at:end].float()).abs().max() <= 2.0 ** -6 * o.abs().max()
        assert (lse2 - lse[:, :, at:end]).abs().max() <= 1e-5
        at = end


def test_prefill_long_against_sampled_rows():
    """A chunk at the end of 131072 positions: the first, the last and some other rows."""
    Lq, Lk, win, sinks = 700, 131072, 4096, 64
    q, k, v = make(1, Lq, Lk, 6, 2, 128, seed=9)
    o, lse = attn_prefill_window(q, k, v, win, sinks)
    for i in (0, 1, 127, 128, 500, 699):
        end = Lk - Lq + i + 1
        at = [*range(sinks), *range(end - win, end)]
        ref = ow.attention(to_np(q[:, i:i + 1]), to_np(k[:, at]), to_np(v[:, at]), len(at), 0)
        check_rows(o[:, i:i + 1], lse[:, :, i:i + 1], ref, 128, str(i))


# ------------------------------------------------------------------ backward

BWD = [
    # B, L, n_q, n_kv, d, W, S
    (1, 1, 1, 1, 64, 1, 0),
    (1, 300, 4, 2, 128, 1, 0),                   # P is the identity: dQ = dK = 0
    (1, 300, 4, 2, 128, 1, 1),
    (2, 333, 4, 1, 64, 100, 3),
    (1, 520, 3, 1, 128, 128, 0),
    (1, 520, 3, 1, 128, 129, 130),
    (1, 1000, 8, 2, 64, 256, 0),
    (1, 1100, 2, 2, 128, 127, 300),
    (1, 400, 6, 2, 128, 400, 5),                 # nothing hidden
    (1, 2100, 2, 1, 64, 50, 1),                  # a sink's tile in many pieces
    (1, 1500, 4, 1, 128, 60, 200),
    (2, 700, 8, 1, 64, 64, 700),                 # every position a sink
]


def check_grads(grads, ref, what=""):
    for name, g, r, e in zip(("dq", "dk", "dv"), grads, *ref):
        err, bound = np.abs(to_np(g) - r), e + 2.0 ** -8 * np.abs(r) + 2.0 ** -60
        assert (err <= bound).all(), (what, name, (err - bound).max(), np.abs(r).max())


def run_backward(q, k, v, win, sinks, seed=1, scale=None, **kw):
    o, lse = attn_prefill_window(q, k, v, win, sinks, scale=scale)
    g = torch.Generator(device="cuda").manual_seed(seed)
    do = torch.randn(q.shape, generator=g, device="cuda").to(torch.bfloat16)
    grads = attn_prefill_window_backward(q, k, v, o, lse, do, win, sinks, scale=scale, **kw)
    assert attn_device_check() == ATTN_OK
    ref = ow.backward(*(to_np(x) for x in (q, k, v, o)), lse.cpu().numpy().astype(np.float64),
                      to_np(do), win, sinks, scale=scale)
    return grads, ref, (o, lse, do)


@pytest.mark.parametrize("case", BWD, ids=str)
def test_backward(case):
    B, L, n_q, n_kv, d, win, sinks = case
    q, k, v = make(B, L, L, n_q, n_kv, d, seed=sum(case[:5]))
    grads, ref, _ = run_backward(q, k, v, win, sinks)
    check_grads(grads, ref, str(case))


def test_backward_random_shapes():
    rng = np.random.default_rng(21)
    for n in range(30):
        n_kv = int(rng.choice([1, 2, 3]))
        n_q = n_kv * int(rng.choice([1, 2, 3, 4, 8]))
        L, d = int(rng.integers(1, 900)), int(rng.choice([64, 128]))
        win, sinks = int(rng.integers(1, 400)), int(rng.choice([0, 1, 4, rng.integers(0, 300)]))
        q, k, v = make(1, L, L, n_q, n_kv, d, seed=n)
        grads, ref, _ = run_backward(q, k, v, win, sinks, seed=n)
        check_grads(grads, ref, str((L, n_q, n_kv, d, win, sinks)))


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.25])
def test_backward_other_scales(scale):
    q, k, v = make(1, 300, 300, 4, 2, 64, seed=15)
    grads, ref, _ = run_backward(q, k, v, 70, 5, scale=scale)
    check_grads(grads, ref, str(scale))


def test_backward_without_a_window_is_the_causal_one():
    q, k, v = make(1, 500, 500, 4, 2, 128, seed=16)
    grads, _, (o, lse, do) = run_backward(q, k, v, 500, 3)
    for a, b in zip(grads, attn_prefill_backward(q, k, v, o, lse, do)):
        assert torch.equal(a, b)


def test_backward_same_bits_again_on_a_used_workspace():
    q, k, v = make(1, 2100, 2100, 2, 1, 64, seed=17)
    grads, _, (o, lse, do) = run_backward(q, k, v, 50, 1)
    size = attn_prefill_window_bwd_workspace_bytes(1, 2100, 2, 1, 64, 50, 1)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        again = attn_prefill_window_backward(q, k, v, o, lse, do, 50, 1, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))


# -------------------------------------------------------------------- decode

STEP = [
    # B, C, n_q, n_kv, lens, W, S
    (3, 333, 10, 5, [333, 100, 0], 64, 4),
    (1, 1, 4, 1, [1], 1, 0),
    (1, 1, 4, 1, [0], 1, 1),
    (5, 600, 4, 4, [127, 128, 129, 385, 600], 128, 0),
    (5, 600, 4, 4, [127, 128, 129, 385, 600], 129, 127),
    (4, 2000, 8, 1, [2000, 1, 1999, 640], 1, 1),
    (2, 2000, 12, 1, [2000, 777], 1000, 900),            # sinks up to the window
    (2, 2500, 32, 2, [2500, 1111], 500, 2),
    (1, 40000, 36, 6, [39999], 4096, 130),
    (6, 700, 16, 8, [0, 0, 0, 5, 0, 0], 3, 3),
    (3, 300, 8, 2, [300, 299, 1], 10 ** 12, 10 ** 12),   # nothing hidden
    (40, 260, 14, 2, [(37 * i) % 261 for i in range(40)], 50, 7),
    (300, 140, 4, 2, [(53 * i) % 141 for i in range(300)], 30, 4),
]


def make_step(B, C, n_q, n_kv, lens, win, sinks, seed=0):
    """Inputs of a step with NaN and infinities wherever no token looks."""
    q, k, v = make(B, 1, C, n_q, n_kv, 128, seed=seed)
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    at, end = torch.arange(C, device="cuda")[None], lens.long()[:, None].clamp(0, C)
    hidden = (at >= end) | ((at < end - win) & (at >= sinks))
    k[hidden], v[hidden] = float("nan"), float("inf")
    return q, k, v, lens


@pytest.mark.parametrize("case", STEP, ids=lambda c: "B%d_C%d_q%d_kv%d_W%d_S%d" % (c[:4] + c[5:]))
def test_decode(case):
    q, k, v, lens = make_step(*case, seed=case[0] + case[1])
    o, lse = attn_decode_window(q, k, v, lens, *case[5:])
    assert attn_device_check() == ATTN_OK
    ref = ow.decode_rows(to_np(q), to_np(k), to_np(v), lens.tolist(), *case[5:])
    check_rows(o, lse, ref, 128, str(case[:4]))


def test_decode_random_shapes():
    rng = np.random.default_rng(22)
    for n in range(40):
        n_kv = int(rng.choice([1, 2, 3, 5]))
        n_q = n_kv * int(rng.choice([1, 2, 4, 7, 8, 16]))
        B, C = int(rng.integers(1, 9)), int(rng.integers(1, 1200))
        win, sinks = int(rng.integers(1, 600)), int(rng.choice([0, 1, 4, rng.integers(0, 500)]))
        lens = [int(x) for x in rng.integers(-2, C + 3, B)]
        q, k, v, lens = make_step(B, C, n_q, n_kv, lens, win, sinks, seed=n)
        o, lse = attn_decode_window(q, k, v, lens, win, sinks)
        ref = ow.decode_rows(to_np(q), to_np(k), to_np(v), lens.tolist(), win, sinks)
        check_rows(o, lse, ref, 128, str((B, C, n_q, n_kv, win, sinks)))
    assert attn_device_check() == ATTN_OK


def test_decode_without_a_window_is_the_ragged_one():
    q, k, v, lens = make_step(3, 900, 8, 2, [900, 333, 5], 900, 0, seed=30)
    o, lse = attn_decode_window(q, k, v, lens, 900)
    o2, lse2 = attn_decode_ragged(q, k, v, lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_is_the_last_row_of_a_prefill():
    q, k, v = make(2, 500, 500, 8, 2, 128, seed=31)
    o, lse = attn_prefill_window(q, k, v, 90, 11)
    lens = torch.full((2,), 500, dtype=torch.int32, device="cuda")
    o2, lse2 = attn_decode_window(q[:, -1:].contiguous(), k, v, lens, 90, 11)
    assert (lse2 - lse[:, :, -1:]).abs().max() <= 1e-5
    assert (o2.float() - o[:, -1:].float()).abs().max() <= 2.0 ** -6 * o2.abs().max()


def test_decode_same_bits_again_and_one_workspace():
    size = attn_decode_window_workspace_bytes(4, 3000, 8, 2, window=300, sinks=5)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    q, k, v, lens = make_step(4, 3000, 8, 2, [3000, 17, 0, 2222], 300, 5, seed=32)
    first = attn_decode_window(q, k, v, lens, 300, 5, workspace=ws)
    for _ in range(3):
        again = attn_decode_window(q, k, v, lens, 300, 5, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
