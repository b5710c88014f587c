"""Key weights of rows that have none: an lse of -inf marks a row without keys, as in
a batch padded to one length, and such a row adds nothing whatever its query holds.
The tolerance is that of test_gpu_key_weights (whose check knows rows of -inf)."""

import pytest

import test_gpu_key_weights as weights
from causal_gqa_prefill_gb300 import ATTN_OK, attn_device_check, attn_key_weights

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


CASES = [
    # B, Lq, Lk, n_q, n_kv, d
    (2, 400, 400, 8, 2, 128),
    (2, 401, 900, 6, 1, 64),           # g = 6: 126 of 128 rows; the last step shares rows
    (1, 300, 300, 3, 3, 128),
    (2, 30, 400, 8, 2, 128),           # few rows: 120 columns
    (2, 32, 400, 8, 2, 64),            # 128 columns, none to spare
    (1, 7, 200, 6, 2, 128),            # 21 columns
    (1, 256, 256, 1, 1, 64),           # 256 columns in one buffer
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_%dx%d_q%d_kv%d_d%d" % c)
def test_padded_rows_add_nothing(case, causal):
    """Sequences padded at their end and at their start, single heads' rows too: the
    same bits whatever stands in the padding."""
    q, k, lse = weights.inputs(*case, causal, seed=sum(case))
    B, Lq, g = case[0], case[1], case[3] // case[4]
    lse[0, :, Lq - Lq // 3:] = -INF
    lse[B - 1, :, :Lq // 5] = -INF
    lse[0, g - 1, Lq // 2] = -INF
    want = attn_key_weights(q, k, lse, causal=causal)
    weights.check(q, k, lse, want, causal, what=str(case))
    none = (lse == -INF).transpose(1, 2)
    assert none.any() and not none.all()
    for bad in (NAN, INF, -INF):
        padded = q.clone()
        padded[none] = bad
        got = attn_key_weights(padded, k, lse, causal=causal)
        assert torch.equal(got, want), bad
    assert attn_device_check() == ATTN_OK


@pytest.mark.parametrize("Lq", [400, 30])
def test_infinite_keys_of_padded_rows(Lq):
    """A key that is infinite has no number for a weight in the rows that it belongs
    to, and none at all from rows without keys."""
    q, k, lse = weights.inputs(1, Lq, 400, 4, 2, 128, True, seed=3)
    k[0, 390, 1, 5] = INF
    lse[0, 2:] = -INF
    got = attn_key_weights(q, k, lse)
    assert (got[0, 1] == 0).all() and (got[0, 0] > 0).all()
    lse[0, 2, Lq - 1] = 3.0                          # one row that sees the key
    got = attn_key_weights(q, k, lse)
    assert not torch.isfinite(got[0, 1, 390]) or got[0, 1, 390] == 0
    assert torch.isfinite(got[0, 1, :390]).all() and (got[0, 1, :390] > 0).all()


@pytest.mark.parametrize("Lq", [400, 30])
def test_other_values_of_lse(Lq):
    """Only -inf means no row: +inf is a softmax whose sum is infinite (a finite score's
    weight is 0, an infinite one's NaN), the lowest finite value one that has overflowed,
    and NaN reaches what the row sees."""
    q, k, lse = weights.inputs(1, Lq, 400, 4, 2, 128, True, seed=4)
    good = attn_key_weights(q, k, lse)
    row, at = 11, 400 - Lq + 11
    others = lse.clone()
    others[0, 1, row] = -INF
    rest = attn_key_weights(q, k, others)
    bad = lse.clone()
    bad[0, 1, row] = INF
    assert torch.equal(attn_key_weights(q, k, bad), rest)
    towards, inf_key = q.clone(), k.clone()
    towards[..., 0] = towards[..., 0].abs() + 0.125
    inf_key[0, at, 0, 0] = INF
    assert torch.isnan(attn_key_weights(towards, inf_key, bad)).nonzero().tolist() == [[0, 0, at]]
    for value in (torch.finfo(torch.float32).min, NAN):
        bad[0, 1, row] = value
        got = attn_key_weights(q, k, bad)
        assert not torch.isfinite(got[0, 0, :at + 1]).any()
        assert torch.equal(got[0, 0, at + 1:], good[0, 0, at + 1:])
        assert torch.equal(got[0, 1], good[0, 1])
