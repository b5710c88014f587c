"""Attention behind a sliding window with sinks, on the CPU: the fp64 reference
against brute force, differences and the unwindowed reference, and what the
calls refuse before any CUDA call."""

import math

import numpy as np
import pytest

import causal_gqa_prefill_gb300 as cg
import oracle
from oracle import window as ow

INVALID, UNSUPPORTED = cg.ATTN_ERR_INVALID_ARG, cg.ATTN_ERR_UNSUPPORTED


def _draw(B, Lq, Lk, n_q, n_kv, d, seed=0):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((B, Lq, n_q, d)), rng.standard_normal((B, Lk, n_kv, d)),
            rng.standard_normal((B, Lk, n_kv, d)))


CASES = [(5, 9, 3, 2), (9, 9, 1, 0), (9, 9, 20, 4), (3, 12, 2, 12), (7, 7, 3, 7), (1, 6, 2, 1)]


@pytest.mark.parametrize("Lq,Lk,W,S", CASES)
def test_forward_against_one_key_at_a_time(Lq, Lk, W, S):
    q, k, v = _draw(2, Lq, Lk, 4, 2, 8)
    o, lse, _, _ = ow.attention(q, k, v, W, S, scale=0.4)
    for b in range(2):
        for h in range(4):
            for i in range(Lq):
                p = i + Lk - Lq
                js = [j for j in range(Lk) if j <= p and (p - j < W or j < S)]
                e = [math.exp(0.4 * math.fsum(q[b, i, h] * k[b, j, h // 2])) for j in js]
                total = math.fsum(e)
                ref = sum(x * v[b, j, h // 2] for x, j in zip(e, js)) / total
                assert abs(lse[b, h, i] - math.log(total)) <= 1e-12
                assert np.abs(o[b, i, h] - ref).max() <= 1e-12


def test_a_wide_window_hides_nothing():
    q, k, v = _draw(1, 6, 10, 2, 1, 8, seed=1)
    ref = oracle.attention(q, k, v, causal=True)
    for W, S in ((10, 0), (99, 5), (1, 10), (3, 7)):
        o, lse, _, _ = ow.attention(q, k, v, W, S)
        assert np.abs(o - ref[0]).max() <= 1e-13 and np.abs(lse - ref[1]).max() <= 1e-13


def test_keys_that_no_row_sees_do_not_matter():
    q, k, v = _draw(1, 4, 20, 2, 1, 8, seed=2)
    o, lse, _, _ = ow.attention(q, k, v, 3, 2)
    k[:, 2:14], v[:, 2:14] = np.nan, np.inf
    o2, lse2, _, _ = ow.attention(q, k, v, 3, 2)
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("W,S", [(3, 0), (2, 2), (50, 0), (1, 3)])
def test_backward_against_differences(W, S):
    q, k, v = _draw(1, 7, 7, 2, 1, 4, seed=3)
    g = np.random.default_rng(4).standard_normal(q.shape)
    o, lse, _, _ = ow.attention(q, k, v, W, S)
    grads, _ = ow.backward(q, k, v, o, lse, g, W, S)
    for x, dx in zip((q, k, v), grads):
        for at in np.ndindex(x.shape):
            old, eps = x[at], 1e-5
            x[at] = old + eps
            up = (ow.attention(q, k, v, W, S)[0] * g).sum()
            x[at] = old - eps
            down = (ow.attention(q, k, v, W, S)[0] * g).sum()
            x[at] = old
            assert abs((up - down) / (2 * eps) - dx[at]) <= 1e-8


def test_backward_without_a_window_is_the_plain_one():
    q, k, v = _draw(2, 6, 6, 4, 2, 8, seed=5)
    g = np.random.default_rng(6).standard_normal(q.shape)
    o, lse, _, _ = ow.attention(q, k, v, 6, 0)
    grads, _ = ow.backward(q, k, v, o, lse, g, 6, 0)
    for a, r in zip(grads, oracle.attention_backward(q, k, v, g, causal=True)):
        assert np.abs(a - r).max() <= 1e-12


def test_decode_is_the_last_row():
    q, k, v = _draw(3, 1, 9, 4, 2, 8, seed=7)
    o, lse, _, _ = ow.decode_rows(q, k, v, [9, 4, 0], 3, 1)
    ref = ow.attention(q[1:2], k[1:2, :4], v[1:2, :4], 3, 1)
    assert np.array_equal(o[1], ref[0][0]) and np.array_equal(lse[1], ref[1][0])
    assert not o[2].any() and (lse[2] == -np.inf).all()


# ------------------------------------------------------------------ refusals

FAKE = 1 << 20   # 16-byte aligned, never dereferenced: each call fails validation first


@pytest.fixture(scope="module", autouse=True)
def _library():
    from causal_gqa_prefill_gb300 import build
    build.build()


FWD = [(dict(q=0), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(v=FAKE + 8), INVALID),
       (dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
       (dict(B=0), INVALID), (dict(Lq=0), INVALID), (dict(Lq=129), INVALID),
       (dict(n_q=5), INVALID), (dict(scale=math.nan), INVALID), (dict(d_h=96), UNSUPPORTED),
       (dict(Lk=1 << 31, Lq=1), UNSUPPORTED), (dict(B=1 << 40), UNSUPPORTED)]


@pytest.mark.parametrize("args,expect", FWD)
def test_forward_refusals(args, expect):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, B=1, Lq=128, Lk=128, n_q=4, n_kv=2, d_h=128,
             window=16, sinks=2, scale=0.125)
    a.update(args)
    assert cg.attn_prefill_window_fwd(**a, stream=0) == expect


BWD = [(dict(dout=0), INVALID), (dict(dk=FAKE + 2), INVALID), (dict(window=0), INVALID),
       (dict(sinks=-3), INVALID), (dict(L=0), INVALID), (dict(n_kv=3), INVALID),
       (dict(scale=math.inf), INVALID), (dict(d_h=32), UNSUPPORTED), (dict(L=1 << 31), UNSUPPORTED),
       (dict(workspace_bytes=100), INVALID), (dict(workspace=FAKE + 4), INVALID)]


@pytest.mark.parametrize("args,expect", BWD)
def test_backward_refusals(args, expect):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE,
             workspace=FAKE, workspace_bytes=1 << 40, B=1, L=128, n_q=4, n_kv=2, d_h=128, window=16,
             sinks=2, scale=0.125)
    a.update(args)
    assert cg.attn_prefill_window_bwd(**a, stream=0) == expect


def test_backward_workspace():
    size = cg.attn_prefill_window_bwd_workspace_bytes
    rows = cg.attn_prefill_bwd_workspace_bytes(2, 4096, 8, 2, 128)
    assert size(2, 4096, 8, 2, 128, 256, 0) == rows                 # no sinks: no parts
    assert size(2, 4096, 8, 2, 128, 4096, 9) == rows                # nothing hidden: no parts
    parts = size(2, 4096, 8, 2, 128, 256, 9) - rows
    assert parts > 0 and parts % (2 * 2 * 2 * 128 * 128 * 4) == 0   # whole tiles of dV and dK
    # two CTAs per SM or so bound the parts, whatever the length
    assert size(1, 1 << 20, 8, 8, 128, 16, 4) - cg.attn_prefill_bwd_workspace_bytes(
        1, 1 << 20, 8, 8, 128) <= 304 * 2 * 128 * 128 * 4
    for bad in ((0, 64, 8, 2, 128, 4, 0), (1, 64, 8, 3, 128, 4, 0), (1, 64, 8, 2, 96, 4, 0),
                (1, 64, 8, 2, 64, 0, 0), (1, 64, 8, 2, 64, 4, -1), (1, 1 << 31, 8, 2, 64, 4, 0)):
        assert size(*bad) == -1


STEP = [(dict(lens=0), INVALID), (dict(lens=FAKE + 2), INVALID), (dict(window=0), INVALID),
        (dict(sinks=-1), INVALID), (dict(C=0), INVALID), (dict(d_h=64), UNSUPPORTED),
        (dict(n_q=34), UNSUPPORTED), (dict(C=1 << 31), UNSUPPORTED),
        (dict(workspace_bytes=64), INVALID), (dict(scale=math.nan), INVALID)]


@pytest.mark.parametrize("args,expect", STEP)
def test_decode_refusals(args, expect):
    a = dict(q=FAKE, k=FAKE, v=FAKE, lens=FAKE, o=FAKE, lse=FAKE, workspace=FAKE,
             workspace_bytes=1 << 40, B=1, C=128, n_q=4, n_kv=2, d_h=128, window=16, sinks=2,
             scale=0.125)
    a.update(args)
    assert cg.attn_decode_window_fwd(**a, stream=0) == expect


def test_decode_workspace_follows_what_is_seen():
    size = cg.attn_decode_window_workspace_bytes
    whole = cg.attn_decode_ragged_workspace_bytes(1, 1 << 17, 8, 2)
    assert size(1, 1 << 17, 8, 2, window=128) < whole
    assert size(1, 1 << 17, 8, 2, window=1 << 17) == whole
    assert size(1, 100, 8, 2, window=1 << 40) > 0
    assert size(1, 100, 8, 2, window=0) == size(1, 100, 8, 2, window=5, sinks=-1) == -1


@pytest.mark.parametrize("window,sinks,error", [(0, 0, ValueError), (-1, 0, ValueError),
                                                (4, -1, ValueError), (2.5, 0, TypeError),
                                                (4, None, TypeError)])
def test_python_refuses_windows(window, sinks, error):
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(error):
        cg.attn_prefill_window(x, x, x, window, sinks)
    with pytest.raises(error):
        cg.attn_prefill_window_backward(x, x, x, x, x, x, window, sinks)
    with pytest.raises(error):
        cg.attn_decode_window(x, x, x, x, window, sinks)


def test_python_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: cg.attn_prefill_window(x, x, x, 2),
                 lambda: cg.attn_prefill_window_backward(x, x, x, x, x, x, 2),
                 lambda: cg.attn_decode_window(x[:, :1], x, x, x, 2)):
        with pytest.raises(TypeError, match="CUDA"):
            call()
