"""Windowed forward and gradients with more work units than SMs: CTAs that walk several
units, whose key lists differ in length, with what is brought in early for the next.

Units: a forward one is a pair of 128-row tiles of a K/V head's query heads, one of dQ a
128-row tile of one query head; both are dealt out in rounds of the SM count, left to
right and back again. Every case has two to four rounds and a last one that is not full.
Tolerances: test_gpu_window's.
"""

import numpy as np
import pytest

from causal_gqa_prefill_gb300 import (ATTN_OK, attn_device_check, attn_prefill_window,
                                      attn_prefill_window_backward)
from causal_gqa_prefill_gb300 import workloads as W
from gpu_common import to_np
from oracle import window as ow

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SMS = 152


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def tiles(n):
    return -(-n // 128)


def several_rounds(units):
    return units > SMS and units % SMS


CASES = [
    # B, Lq, Lk, n_q, n_kv, W, S
    (2, 1500, 1500, 24, 3, 60, 0),               # 288 units
    (2, 1500, 1500, 24, 3, 400, 17),
    (2, 1500, 1500, 24, 3, 129, 300),            # sinks of three tiles
    (2, 1500, 1500, 24, 3, 1200, 1),             # lists of one tile to eleven
    (4, 700, 700, 24, 24, 128, 5),               # one head a group: 288
    (3, 900, 900, 21, 7, 1, 2),                  # three heads a group: 252
    (2, 1300, 1300, 20, 4, 256, 1300),           # every position a sink: 224
    (1, 2000, 2000, 48, 6, 33, 0),               # 384
    (2, 1100, 1777, 24, 3, 250, 40),             # chunks: 216
    (9, 300, 2500, 16, 8, 1000, 130),            # 216
    (4, 600, 1601, 16, 8, 90, 0),                # 160
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_prefill(case, d):
    B, Lq, Lk, n_q, n_kv, win, sinks = case
    assert several_rounds(B * n_kv * -(-(n_q // n_kv) * tiles(Lq) // 2))
    q, k, v = W.make_inputs(W.custom(B, Lq, n_q, n_kv, d, Lk=Lk), "cuda", seed=win + sinks + d)
    o, lse = attn_prefill_window(q, k, v, win, sinks)
    assert attn_device_check() == ATTN_OK
    o_r, lse_r, o_abs, s_abs = ow.attention(to_np(q), to_np(k), to_np(v), win, sinks)
    err = np.abs(to_np(o) - o_r)
    assert (err <= 2.0 ** -8 * ((1 + 2.0 ** -6) * o_abs + np.abs(o_r))).all()
    err = np.abs(lse.cpu().numpy().astype(np.float64) - lse_r)
    assert (err <= (d + 2) * 2.0 ** -24 * s_abs + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse_r)).all()
    again = attn_prefill_window(q, k, v, win, sinks)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", [(1, 1500, 24, 3, 60, 0), (1, 1500, 24, 3, 400, 17),
                                  (2, 1100, 24, 3, 129, 300), (1, 1500, 24, 3, 1200, 1),
                                  (2, 700, 24, 24, 128, 5), (3, 900, 21, 7, 2, 2),
                                  (1, 1300, 20, 4, 256, 1300)], ids=str)
def test_backward(case, d):
    B, L, n_q, n_kv, win, sinks = case
    assert several_rounds(B * n_q * tiles(L))
    q, k, v = W.make_inputs(W.custom(B, L, n_q, n_kv, d), "cuda", seed=win + sinks + d + 1)
    o, lse = attn_prefill_window(q, k, v, win, sinks)
    g = torch.Generator(device="cuda").manual_seed(L)
    do = torch.randn(q.shape, generator=g, device="cuda").to(torch.bfloat16)
    grads = attn_prefill_window_backward(q, k, v, o, lse, do, win, sinks)
    assert attn_device_check() == ATTN_OK
    ref = ow.backward(*(to_np(x) for x in (q, k, v, o)), lse.cpu().numpy().astype(np.float64),
                      to_np(do), win, sinks)
    for name, x, r, e in zip(("dq", "dk", "dv"), grads, *ref):
        err, bound = np.abs(to_np(x) - r), e + 2.0 ** -8 * np.abs(r) + 2.0 ** -60
        assert (err <= bound).all(), (name, (err - bound).max(), np.abs(r).max())
    again = attn_prefill_window_backward(q, k, v, o, lse, do, win, sinks)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
