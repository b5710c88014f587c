"""Which rows of a windowed forward something not finite reaches.

A unit of work multiplies whole tiles of 128 keys from the one that holds the first
position of its first row's window on, for up to 256 rows, each up to the tile of its own
128-row tile's last position. So V at position j meets the rows from j - 254 (j - 127 where
rows and keys begin together) to j + W + 381, and for a sink all later ones, whether they
see it or not; K at j only decides over scores that rows see. Rows outside keep their
bits (V) or stay within the forward's bound of what they were without it (K: warps
rescale together).
"""

import numpy as np
import pytest

from causal_gqa_prefill_gb300 import ATTN_OK, attn_device_check, attn_prefill_window
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


CASES = [
    # Lq, Lk, n_q, n_kv, d, W, S
    (1500, 1500, 1, 1, 128, 130, 0),       # a unit is two neighbouring tiles of the one head
    (1500, 1500, 1, 1, 64, 1, 0),
    (1500, 1500, 4, 1, 128, 300, 9),
    (1100, 1777, 2, 2, 64, 129, 0),        # rows and keys do not begin together
    (1000, 1403, 3, 1, 128, 40, 200),
    (1500, 1500, 2, 1, 128, 128, 5),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_reach(case):
    Lq, Lk, n_q, n_kv, d, win, sinks = case
    q, k, v = W.make_inputs(W.custom(1, Lq, n_q, n_kv, d, Lk=Lk), "cuda", seed=win)
    o, lse = attn_prefill_window(q, k, v, win, sinks)
    ref, lse_ref, o_abs, s_abs = ow.attention(to_np(q), to_np(k), to_np(v), win, sinks)
    first = Lk - Lq
    p = np.arange(first, Lk)
    for j in (0, 1, 127, 128, 255, 256, 500, first, first + 300, first + 511, Lk - 1):
        if j >= sinks and j < first - win + 1:
            continue                       # no row sees it
        sees = (j <= p) & ((j > p - win) | (j < sinks))
        meets = (p >= j - 254) & ((p <= j + win + 381) | (j < sinks))
        head = slice(0, n_q // n_kv)       # of the first K/V head
        for bad in (float("nan"), float("inf")):
            v2 = v.clone()
            v2[:, j, 0] = bad
            o2, lse2 = attn_prefill_window(q, k, v2, win, sinks)
            assert torch.equal(lse2, lse)
            seen = to_np(o2)[0, sees][:, head]
            assert not np.isfinite(seen).any()
            keep = torch.from_numpy(~meets).cuda()
            assert torch.equal(o2[:, keep], o[:, keep])
            assert torch.equal(o2[:, :, n_q // n_kv:], o[:, :, n_q // n_kv:])
        k2 = k.clone()
        k2[:, j, 0] = float("nan")
        o2, lse2 = attn_prefill_window(q, k2, v, win, sinks)
        assert np.isnan(to_np(o2)[0, sees][:, head]).all() and lse2[0, head][:, torch.from_numpy(sees).cuda()].isnan().all()
        err = np.abs(to_np(o2) - ref)[0, ~sees]
        bound = (2.0 ** -8 * ((1 + 2.0 ** -6) * o_abs + np.abs(ref)))[0, ~sees]
        assert (err <= bound).all()
        err = np.abs(lse2.cpu().numpy().astype(np.float64) - lse_ref)[0][:, ~sees]
        bound = ((d + 2) * 2.0 ** -24 * s_abs + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse_ref))[0][:, ~sees]
        assert (err <= bound).all()
    assert attn_device_check() == ATTN_OK
