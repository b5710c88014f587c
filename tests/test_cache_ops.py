"""The cache operators without a GPU: what the library refuses before its first
CUDA call, what the Python calls refuse, and the oracle against values worked
out by hand and against the attention oracle."""

import math

import numpy as np
import pytest

import causal_gqa_prefill_gb300 as cg
import oracle
from causal_gqa_prefill_gb300 import build

BAD, UNSUP = cg.ATTN_ERR_INVALID_ARG, cg.ATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return cg.load_library()


# addresses that nothing reads: every call below fails its checks first
def _at(i):
    return (1 << 40) + (i << 36)


def _call(fn, order, base, change):
    a = dict(base)
    a.update(change)
    return fn(*[a[n] for n in order], stream=0)


# --------------------------------------------------------------- key weights

WEIGHTS_ORDER = ("q k lse weights workspace workspace_bytes B Lq Lk n_q n_kv d_h causal accumulate "
                 "scale").split()
WEIGHTS_BASE = dict(q=_at(0), k=_at(1), lse=_at(2), weights=_at(3), workspace=_at(4),
                    workspace_bytes=1 << 20, B=2, Lq=300, Lk=500, n_q=8, n_kv=2, d_h=128, causal=1,
                    accumulate=0, scale=0.1)


@pytest.mark.parametrize("change,expect", [
    (dict(q=0), BAD), (dict(k=0), BAD), (dict(lse=0), BAD), (dict(weights=0), BAD),
    (dict(workspace=0), BAD), (dict(workspace_bytes=1000), BAD), (dict(B=0), BAD),
    (dict(Lq=0), BAD), (dict(Lq=501), BAD), (dict(n_q=7), BAD), (dict(n_kv=0), BAD),
    (dict(causal=2), BAD), (dict(accumulate=-1), BAD), (dict(scale=math.nan), BAD),
    (dict(q=_at(0) + 8), BAD), (dict(lse=_at(2) + 2), BAD), (dict(workspace=_at(4) + 4), BAD),
    (dict(d_h=96), UNSUP), (dict(n_q=258), UNSUP), (dict(Lk=1 << 31), UNSUP),
    (dict(Lq=1 << 30, Lk=1 << 30), UNSUP),
], ids=str)
def test_key_weights_refuse(change, expect):
    assert _call(cg.attn_key_weights_fwd, WEIGHTS_ORDER, WEIGHTS_BASE, change) == expect


def test_key_weights_workspace():
    size = cg.attn_key_weights_workspace_bytes
    assert size(1, 100, 100, 8, 2) == size(3, 1, 100000, 128, 1, 64) > 0
    for bad in ((0, 1, 1, 1, 1), (1, 2, 1, 1, 1), (1, 1, 1, 3, 2), (1, 1, 1, 129, 1),
                (1, 1, 1, 1, 1, 32)):
        assert size(*bad) == -1, bad


# ------------------------------------------------------------- ragged decode

RAGGED_ORDER = ("q k v lens weights o lse workspace workspace_bytes B C n_q n_kv d_h "
                "scale").split()


def _ragged_base():
    need = cg.attn_decode_ragged_workspace_bytes(2, 1000, 8, 2, weighted=True)
    return dict(q=_at(0), k=_at(1), v=_at(2), lens=_at(3), weights=_at(4), o=_at(5), lse=_at(6),
                workspace=_at(7), workspace_bytes=need, B=2, C=1000, n_q=8, n_kv=2, d_h=128,
                scale=0.1)


@pytest.mark.parametrize("change,expect", [
    (dict(q=0), BAD), (dict(k=0), BAD), (dict(v=0), BAD), (dict(lens=0), BAD), (dict(o=0), BAD),
    (dict(lse=0), BAD), (dict(workspace=0), BAD), (dict(B=0), BAD), (dict(C=0), BAD),
    (dict(n_q=7), BAD), (dict(n_kv=0), BAD), (dict(scale=math.nan), BAD),
    (dict(scale=math.inf), BAD), (dict(k=_at(1) + 8), BAD), (dict(lens=_at(3) + 2), BAD),
    (dict(weights=_at(4) + 1), BAD), (dict(workspace=_at(7) + 4), BAD), (dict(d_h=64), UNSUP),
    (dict(n_q=34), UNSUP), (dict(C=1 << 31), UNSUP), (dict(B=1 << 25), UNSUP),
], ids=str)
def test_ragged_decode_refuses(change, expect):
    assert _call(cg.attn_decode_ragged_fwd, RAGGED_ORDER, _ragged_base(), change) == expect


def test_ragged_decode_workspace():
    size = cg.attn_decode_ragged_workspace_bytes
    plain, weighted = size(2, 1000, 8, 2), size(2, 1000, 8, 2, weighted=True)
    assert weighted == plain + 2 * 8 * 1024 * 4           # scores, positions in whole tiles
    small = dict(workspace_bytes=weighted - 1)
    assert _call(cg.attn_decode_ragged_fwd, RAGGED_ORDER, _ragged_base(), small) == BAD
    small = dict(workspace_bytes=plain - 1, weights=0)
    assert _call(cg.attn_decode_ragged_fwd, RAGGED_ORDER, _ragged_base(), small) == BAD
    for bad in ((0, 10, 8, 2), (1, 0, 8, 2), (1, 10, 8, 3), (1, 10, 34, 2), (1, 10, 8, 2, 64)):
        assert size(*bad) == -1, bad


# -------------------------------------------------------------- shared prefix

SHARED_ORDER = ("q prefix_k prefix_v k v lens o lse workspace workspace_bytes B P C n_q n_kv d_h "
                "scale").split()


def _shared_base():
    need = cg.attn_decode_shared_workspace_bytes(40, 1000, 300, 8, 2)
    return dict(q=_at(0), prefix_k=_at(1), prefix_v=_at(2), k=_at(3), v=_at(4), lens=_at(5),
                o=_at(6), lse=_at(7), workspace=_at(8), workspace_bytes=need, B=40, P=1000, C=300,
                n_q=8, n_kv=2, d_h=128, scale=0.1)


@pytest.mark.parametrize("change,expect", [
    (dict(q=0), BAD), (dict(prefix_k=0), BAD), (dict(prefix_v=0), BAD), (dict(k=0), BAD),
    (dict(v=0), BAD), (dict(lens=0), BAD), (dict(o=0), BAD), (dict(lse=0), BAD),
    (dict(workspace=0), BAD), (dict(B=0), BAD), (dict(P=0), BAD), (dict(C=0), BAD),
    (dict(n_q=9), BAD), (dict(n_kv=-1), BAD), (dict(scale=math.inf), BAD),
    (dict(prefix_k=_at(1) + 8), BAD), (dict(lens=_at(5) + 1), BAD),
    (dict(workspace=_at(8) + 8), BAD), (dict(d_h=64), UNSUP), (dict(n_q=34), UNSUP),
    (dict(P=1 << 31), UNSUP), (dict(C=1 << 31), UNSUP), (dict(B=1 << 25), UNSUP),
], ids=str)
def test_shared_decode_refuses(change, expect):
    assert _call(cg.attn_decode_shared_fwd, SHARED_ORDER, _shared_base(), change) == expect


def test_shared_decode_workspace():
    base = _shared_base()
    small = dict(workspace_bytes=base["workspace_bytes"] - 1)
    assert _call(cg.attn_decode_shared_fwd, SHARED_ORDER, base, small) == BAD
    size = cg.attn_decode_shared_workspace_bytes
    for bad in ((0, 1, 1, 1, 1), (1, 0, 1, 1, 1), (1, 1, 0, 1, 1), (1, 1, 1, 3, 2),
                (1, 1, 1, 17, 1), (1, 1, 1, 1, 1, 64)):
        assert size(*bad) == -1, bad


# ------------------------------------------------------------------ eviction

EVICT_ORDER = ("k v weights lens k_out v_out weights_out lens_out index B C C_out budget recent "
               "n_kv d_h elem_bytes").split()
EVICT_BASE = dict(k=_at(0), v=_at(1), weights=_at(2), lens=_at(3), k_out=_at(4), v_out=_at(5),
                  weights_out=_at(6), lens_out=_at(7), index=_at(8), B=2, C=1000, C_out=300,
                  budget=256, recent=32, n_kv=2, d_h=128, elem_bytes=2)
K_BYTES = 2 * 1000 * 2 * 128 * 2


@pytest.mark.parametrize("change,expect", [
    (dict(k=0), BAD), (dict(v=0), BAD), (dict(weights=0), BAD), (dict(lens=0), BAD),
    (dict(k_out=0), BAD), (dict(v_out=0), BAD), (dict(weights_out=0), BAD),
    (dict(lens_out=0), BAD), (dict(index=0), BAD), (dict(B=0), BAD), (dict(C=0), BAD),
    (dict(budget=0), BAD), (dict(recent=-1), BAD), (dict(recent=257), BAD), (dict(C_out=255), BAD),
    (dict(elem_bytes=4), BAD), (dict(n_kv=0), BAD), (dict(k=_at(0) + 8), BAD),
    (dict(index=_at(8) + 2), BAD), (dict(d_h=96), UNSUP), (dict(n_kv=129), UNSUP),
    (dict(C=1 << 31), UNSUP), (dict(B=1 << 24), UNSUP),
    # outputs that overlap inputs or each other
    (dict(k_out=_at(0)), BAD), (dict(k_out=_at(0) + K_BYTES - 16), BAD), (dict(v_out=_at(4)), BAD),
    (dict(lens_out=_at(3)), BAD), (dict(weights_out=_at(2) + 4), BAD), (dict(index=_at(7) + 4), BAD),
], ids=str)
def test_evict_refuses(change, expect):
    assert _call(cg.attn_cache_evict, EVICT_ORDER, EVICT_BASE, change) == expect


def test_python_calls_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    q, kv = (torch.zeros(1, n, 2, 128, dtype=torch.bfloat16) for n in (1, 8))
    lens = torch.ones(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        cg.attn_decode_ragged(q, kv, kv, lens)
    with pytest.raises(TypeError):
        cg.attn_evict(kv, kv, torch.zeros(1, 2, 8), lens, 4)
    with pytest.raises(TypeError):
        cg.attn_evict(kv.float(), kv, torch.zeros(1, 2, 8), lens, 4)


# ---------------------------------------------------------------- the oracle


def test_oracle_decode_is_the_attention_oracle():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(2, 1, 6, 16)), rng.normal(size=(2, 9, 3, 16)), \
        rng.normal(size=(2, 9, 3, 16))
    o, lse, added, _, _ = oracle.cache.decode_rows(q, k, v, [9, 5])
    for b, n in ((0, 9), (1, 5)):
        o1, l1 = oracle.attention(q[b:b + 1], k[b:b + 1, :n], v[b:b + 1, :n], causal=True)
        assert np.allclose(o[b], o1[0], atol=1e-12) and np.allclose(lse[b], l1[0], atol=1e-12)
    assert np.allclose(added.sum(2), 2.0)                   # every head's weights add up to one
    assert (added[1, :, 5:] == 0).all()
    # a prefix is the same as keys in front of every sequence
    pk, pv = rng.normal(size=(1, 4, 3, 16)), rng.normal(size=(1, 4, 3, 16))
    o2, l2, _, _, _ = oracle.cache.decode_rows(q, k, v, [9, 0], prefix_k=pk, prefix_v=pv)
    for b, n in ((0, 9), (1, 0)):
        o1, l1 = oracle.attention(q[b:b + 1], np.concatenate([pk, k[b:b + 1, :n]], 1),
                                  np.concatenate([pv, v[b:b + 1, :n]], 1), causal=True)
        assert np.allclose(o2[b], o1[0], atol=1e-12) and np.allclose(l2[b], l1[0], atol=1e-12)


def test_oracle_key_weights():
    rng = np.random.default_rng(4)
    q, k = rng.normal(size=(1, 5, 4, 8)), rng.normal(size=(1, 7, 2, 8))
    _, lse = oracle.attention(q, k, k, causal=True)
    w = oracle.cache.key_weights(q, k, lse)
    assert np.allclose(w.sum(2), 5 * 2)                     # a row's weights add up to one
    by_rows = np.zeros_like(w)
    for i in range(5):                                      # each row is a decode step
        by_rows += oracle.cache.decode_rows(q[:, i:i + 1], k, k, [i + 3])[2]
    assert np.allclose(w, by_rows, atol=1e-12)
    lse[0, 1, 2] = -np.inf                                  # a row without keys adds nothing
    less = oracle.cache.key_weights(q, k, lse)
    assert np.allclose(less[0, 0].sum(), 9.0) and np.allclose(less[0, 1], w[0, 1])


def test_oracle_key_weights_of_padded_rows():
    """A row whose lse is -inf adds nothing, whatever its q and the keys hold."""
    rng = np.random.default_rng(5)
    q, k = rng.normal(size=(1, 6, 4, 8)), rng.normal(size=(1, 6, 2, 8))
    _, lse = oracle.attention(q, k, k, causal=True)
    lse[0, 1, 2:4] = lse[0, 2, 5] = -np.inf
    want = oracle.cache.key_weights(q, k, lse)
    for bad in (np.nan, np.inf, -np.inf):
        padded = q.copy()
        padded[0, 2:4, 1] = padded[0, 5, 2] = bad
        with np.errstate(invalid="ignore"):
            assert np.array_equal(oracle.cache.key_weights(padded, k, lse), want), bad


def test_oracle_eviction_by_hand():
    w = np.array([[[3.0, 1.0, np.nan, 1.0, 5.0, 0.0, -0.0, 2.0]]])
    index, lens = oracle.cache.evicted_index(w, [8], 4, 1)
    assert index.tolist() == [[[0, 1, 4, 7]]] and lens.tolist() == [4]   # 1.0 tie: position 1
    index, lens = oracle.cache.evicted_index(w, [7], 6, 0)
    assert index.tolist() == [[[0, 1, 3, 4, 5, 6]]]                      # the NaN goes first
    index, lens = oracle.cache.evicted_index(w, [3], 4, 4)
    assert index.tolist() == [[[0, 1, 2, -1]]] and lens.tolist() == [3]
    index, lens = oracle.cache.evicted_index(w, [8], 3, 3)
    assert index.tolist() == [[[5, 6, 7]]]
    index, lens = oracle.cache.evicted_index(w, [0], 3, 3)
    assert index.tolist() == [[[-1, -1, -1]]] and lens.tolist() == [0]
