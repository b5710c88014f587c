"""What is not a number in one query, key or value of a ragged decode step stays in the
rows and weights that it belongs to: everything else keeps its bits."""

import pytest

from cache_common import make
from causal_gqa_prefill_gb300 import ATTN_OK, attn_decode_ragged, attn_device_check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


LENS = [300, 1, 0, 133, 128, 1500]


def step(q, k, v, lens, acc):
    mine = acc.clone()
    o, lse = attn_decode_ragged(q, k, v, lens, weights=mine)
    assert attn_device_check() == ATTN_OK
    return o[:, 0], lse[..., 0], mine


def compare(good, got, lens, g, nan_rows, nan_out):
    """nan_rows [B, n_q]: rows whose lse is NaN, and whose K/V heads' weights are;
    nan_out [B, n_q, 128]: where the output is NaN."""
    (o, lse, w), (o2, lse2, w2) = good, got
    assert torch.equal(torch.isnan(o2), nan_out)
    assert torch.equal(o2[~nan_out], o[~nan_out])
    assert torch.equal(torch.isnan(lse2), nan_rows)
    assert torch.equal(lse2[~nan_rows], lse[~nan_rows])
    B, n_kv, C = w.shape
    held = torch.arange(C, device="cuda")[None, None] < lens[:, None, None]
    bad = nan_rows.reshape(B, n_kv, g).any(2)[..., None] & held
    assert torch.equal(torch.isnan(w2), bad)
    assert torch.equal(w2[~bad], w[~bad])


@pytest.mark.parametrize("n_q,n_kv", [(8, 2), (6, 6), (32, 2), (24, 8)])
def test_nan_stays_where_it_belongs(n_q, n_kv):
    B, C, g = len(LENS), 1500, n_q // n_kv
    q, k, v, lens, acc = make(B, C, n_q, n_kv, LENS, seed=n_q, junk=False)
    good = step(q, k, v, lens, acc)
    assert all(torch.isfinite(x).all() for x in (good[0], good[2]))
    clean = torch.zeros(B, n_q, dtype=torch.bool, device="cuda")
    none = torch.zeros(B, n_q, 128, dtype=torch.bool, device="cuda")

    rows = clean.clone()                            # queries
    bad = q.clone()
    for b, h, e in ((0, n_q - 1, 7), (1, 0, 0), (5, n_q // 2, 127)):
        bad[b, 0, h, e], rows[b, h] = NAN, True
    bad[2, 0, 1, 0] = NAN                           # a sequence without keys stays 0
    compare(good, step(bad, k, v, lens, acc), lens, g, rows, rows[..., None].expand_as(none))

    rows = clean.clone()                            # keys: at tile ends, alone, last
    bad = k.clone()
    for b, j, u in ((0, 127, n_kv - 1), (1, 0, 0), (3, 132, 0), (4, 127, n_kv - 1), (5, 1024, 0)):
        bad[b, j, u, 3], rows[b, g * u:g * u + g] = NAN, True
    bad[0, 300], bad[2, 0], bad[4, 128] = NAN, INF, NAN      # behind the sequences
    compare(good, step(q, bad, v, lens, acc), lens, g, rows, rows[..., None].expand_as(none))

    out = none.clone()                              # values: one dimension, no weight
    bad = v.clone()
    for b, j, u, e in ((0, 299, 0, 0), (1, 0, n_kv - 1, 127), (5, 255, n_kv - 1, 64)):
        bad[b, j, u, e], out[b, g * u:g * u + g, e] = NAN, True
    bad[0, 300], bad[2, 0], bad[4, 128] = NAN, INF, NAN
    compare(good, step(q, k, bad, lens, acc), lens, g, clean, out)
