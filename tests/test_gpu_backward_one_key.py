"""Gradients of rows that see one key: a softmax of one weight is 1 whatever its score,
so dS = P (dP - D) is 0 and with it what the row gives to dQ and dK, exactly.

A row sees one key at position 0 of a causal call, everywhere behind a window of 1
without sinks, and in a call over one position. Zeros are compared bit by bit (no -0). dV is
the sum of the group's dO in fp32 and rounds to bf16 once: |dV - ref| <= 2^-8 |ref| +
g 2^-23 sum |dO| (the weight is 1 to within 2^-20 and 1 in bf16). The other rows, keys
and gradients: oracle.window.backward's sums and half a bf16 step of the result, as for
every windowed gradient.
"""

import numpy as np
import pytest

from causal_gqa_prefill_gb300 import (ATTN_OK, attn_device_check, attn_prefill,
                                      attn_prefill_backward, attn_prefill_window,
                                      attn_prefill_window_backward)
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


def gradients(B, L, n_q, n_kv, d, window=None, sinks=0, causal=True, seed=0, spoil=None):
    q, k, v = W.make_inputs(W.custom(B, L, n_q, n_kv, d), "cuda", seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    do = torch.randn(q.shape, generator=g, device="cuda").to(torch.bfloat16)
    if spoil:
        spoil(q, k, v, do)
    if window is None:
        o, lse = attn_prefill(q, k, v, causal=causal)
        grads = attn_prefill_backward(q, k, v, o, lse, do, causal=causal)
    else:
        o, lse = attn_prefill_window(q, k, v, window, sinks)
        grads = attn_prefill_window_backward(q, k, v, o, lse, do, window, sinks)
    assert attn_device_check() == ATTN_OK
    return grads, (q, k, v, o, lse, do)


def check_only_dv(grads, do, n_kv):
    dq, dk, dv = grads
    assert not dq.view(torch.int16).any() and not dk.view(torch.int16).any()
    B, L, n_q, d = do.shape
    do = to_np(do).reshape(B, L, n_kv, n_q // n_kv, d)
    ref, size = do.sum(3), np.abs(do).sum(3)
    err = np.abs(to_np(dv) - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + (n_q // n_kv) * 2.0 ** -23 * size).all()


HEADS = [(1, 1), (8, 2), (6, 1)]


@pytest.mark.parametrize("how", [None, "full", (1, 0), (7, 0), (1, 5)], ids=str)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_one_position(heads, d, how):
    kw = dict(causal=how is None) if how in (None, "full") else dict(window=how[0], sinks=how[1])
    grads, (*_, do) = gradients(3, 1, *heads, d, seed=heads[0] + d, **kw)
    check_only_dv(grads, do, heads[1])


@pytest.mark.parametrize("L", [2, 127, 128, 129, 300, 1100])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_window_of_one(heads, d, L):
    grads, (*_, do) = gradients(2, L, *heads, d, window=1, seed=L)
    check_only_dv(grads, do, heads[1])


def test_window_of_one_in_every_round_of_units():
    grads, (*_, do) = gradients(2, 4000, 16, 4, 128, window=1, seed=3)
    check_only_dv(grads, do, 4)


@pytest.mark.parametrize("window,sinks", [(None, 0), (2, 0), (1, 1), (100, 0), (128, 0), (129, 3),
                                          (40, 200), (700, 0)])
@pytest.mark.parametrize("d", [64, 128])
def test_the_first_position(d, window, sinks):
    B, L, n_q, n_kv = 2, 700, 8, 2
    grads, (q, k, v, o, lse, do) = gradients(B, L, n_q, n_kv, d, window, sinks, seed=d + sinks)
    assert not grads[0][:, 0].any() and grads[0][:, 1:].any(-1).all()
    ref = ow.backward(*(to_np(x) for x in (q, k, v, o)), lse.cpu().numpy().astype(np.float64),
                      to_np(do), L if window is None else window, sinks)
    for g, r, e in zip(grads, *ref):
        assert (np.abs(to_np(g) - r) <= e + 2.0 ** -8 * np.abs(r) + 2.0 ** -60).all()


@pytest.mark.parametrize("window", [None, 1, 90])
@pytest.mark.parametrize("d", [64, 128])
def test_what_is_not_a_number_stays(d, window):
    def spoil(q, k, v, do):
        q[1, 0, 3] = float("nan")

    grads, _ = gradients(2, 200, 4, 2, d, window, seed=9, spoil=spoil)
    assert grads[0][1, 0, 3].isnan().all()
    assert not grads[0][0, 0].any() and not grads[0][1, 0, :3].any()
