"""GPU parity of the key weights against the fp64 oracle.

Tolerance. A row's weight exp(s - LSE) is off by the score's fp32 error, at most
(d + 2) 2^-24 scale sum |q_d k_d|, by the roundings of c s - lse2 in the exponent
(its operands and its result: 2^-22 (|s| + |LSE|) covers their half steps and the
factor log2 e) and by 2^-22 of the exponential; 64 additions of a step's columns
and one per range border of a key's steps add 2^-24 each, at most 2^-16 with 152
ranges. The sums are of positive terms, so the relative bound carries over.
"""

import numpy as np
import pytest

import oracle
from causal_gqa_prefill_gb300 import (ATTN_OK, AttnError, attn_device_check, attn_key_weights,
                                      attn_prefill)
from causal_gqa_prefill_gb300 import workloads as W
from gpu_common import to_np

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def rel_bound(q, k, lse, scale):
    d = q.shape[3]
    size = abs(scale) * np.linalg.norm(q, axis=3).max() * np.linalg.norm(k, axis=3).max()
    top = np.abs(lse[np.isfinite(lse)]).max() if np.isfinite(lse).any() else 0.0
    return (d + 2) * 2.0 ** -24 * size + 2.0 ** -22 * (size + top) + 2.0 ** -22 + 2.0 ** -16


def inputs(B, Lq, Lk, n_q, n_kv, d, causal, seed, scale=None):
    w = W.custom(B, Lq, n_q, n_kv, d, causal=causal, Lk=Lk)
    q, k, v = W.make_inputs(w, "cuda", seed=seed)
    _, lse = attn_prefill(q, k, v, causal=causal, scale=scale)
    return q, k, lse


def check(q, k, lse, got, causal=True, scale=None, before=None, what=""):
    qn, kn, ln = to_np(q), to_np(k), lse.cpu().numpy().astype(np.float64)
    scale = q.shape[3] ** -0.5 if scale is None else scale
    ref = oracle.cache.key_weights(qn, kn, ln, causal=causal, scale=scale)
    bound = rel_bound(qn, kn, ln, scale) * ref
    if before is not None:
        ref = ref + before.cpu().numpy().astype(np.float64)
        bound = bound + 2.0 ** -23 * np.abs(ref)
    err = np.abs(got.cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound).all(), (what, (err / np.maximum(bound, 1e-300)).max())


CASES = [
    # B, Lq, Lk, n_q, n_kv, d
    (1, 1, 1, 1, 1, 128),
    (2, 1, 1, 4, 2, 64),
    (1, 256, 256, 4, 1, 64),
    (2, 257, 257, 8, 2, 128),
    (3, 130, 130, 10, 5, 64),          # g = 2
    (1, 700, 700, 6, 1, 128),          # g = 6: 126 of 128 columns
    (1, 500, 500, 7, 1, 64),           # g = 7
    (2, 300, 300, 3, 3, 128),          # g = 1
    (1, 640, 640, 32, 2, 128),         # g = 16
    (1, 90, 90, 71, 1, 64),            # g = 71: one row a step
    (1, 70, 70, 128, 1, 128),          # g = 128
    (1, 1, 1000, 8, 2, 128),           # one row
    (2, 32, 3000, 6, 2, 128),          # the last rows of longer prompts
    (1, 100, 517, 4, 4, 64),
    (2, 128, 640, 12, 4, 128),
    (4, 33, 65, 2, 1, 128),
    (40, 20, 200, 2, 2, 64),           # more units than CTAs
    # up to 256 columns (rows x heads of a group): one tile for all of them
    (1, 64, 900, 8, 2, 128),           # 256
    (2, 32, 1300, 8, 2, 64),           # 128: two Q buffers
    (1, 43, 700, 6, 1, 128),           # 258: one too many
    (3, 33, 40, 4, 1, 128),            # 132, most keys hidden from most rows
    (1, 2, 130, 128, 1, 64),           # 256 of two rows
    (7, 5, 1000, 35, 5, 128),          # 35, heads change inside CTAs' ranges
    (1, 256, 256, 1, 1, 128),
    (30, 3, 64, 8, 8, 64),             # a tile a head, 240 heads
    (1, 1500, 1501, 2, 1, 128),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_%dx%d_q%d_kv%d_d%d" % c)
def test_against_the_oracle(case, causal):
    q, k, lse = inputs(*case, causal, seed=sum(case))
    w = attn_key_weights(q, k, lse, causal=causal)
    assert attn_device_check() == ATTN_OK
    check(q, k, lse, w, causal, what=str(case))
    total = case[0] * case[1] * case[3]                 # every row's weights add up to one
    assert abs(w.double().sum().item() - total) <= 1e-4 * total


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_other_scales(scale):
    q, k, lse = inputs(1, 200, 300, 6, 2, 128, True, seed=4, scale=scale)
    w = attn_key_weights(q, k, lse, scale=scale)
    check(q, k, lse, w, scale=scale, what=str(scale))


def test_chunks_add_up_to_the_whole():
    """A prompt's chunks accumulated into one tensor equal the whole prompt's weights."""
    q, k, lse = inputs(2, 777, 777, 8, 2, 128, True, seed=5)
    whole = attn_key_weights(q, k, lse)
    acc = torch.zeros_like(whole)
    for a, b in ((0, 300), (300, 301), (301, 777)):
        part = acc[..., :b].contiguous()
        before = part.clone()
        args = (q[:, a:b].contiguous(), k[:, :b].contiguous(), lse[..., a:b].contiguous())
        attn_key_weights(*args, weights=part, accumulate=True)
        check(*args, part, before=before, what=str((a, b)))
        acc[..., :b] = part
    assert torch.allclose(acc, whole, rtol=1e-4, atol=0)


def test_rows_without_keys_add_nothing():
    q, k, lse = inputs(1, 300, 300, 4, 2, 128, True, seed=6)
    lse[0, 1, 7] = lse[0, 2, 255:] = -float("inf")
    check(q, k, lse, attn_key_weights(q, k, lse))
    lse[:] = -float("inf")
    assert (attn_key_weights(q, k, lse) == 0).all()


def test_hidden_values_do_not_leak():
    """A NaN key makes its own weight NaN and no other; a NaN query only those of
    the keys it sees."""
    q, k, lse = inputs(1, 400, 400, 4, 2, 128, True, seed=7)
    good = attn_key_weights(q, k, lse)
    bad = k.clone()
    bad[0, 37, 0] = float("nan")
    w = attn_key_weights(q, bad, lse)
    assert torch.isnan(w).nonzero().tolist() == [[0, 0, 37]]
    w[0, 0, 37] = good[0, 0, 37]
    assert torch.equal(w, good)
    bad = q.clone()
    bad[0, 100, 3] = float("nan")
    w = attn_key_weights(bad, k, lse)
    assert torch.isnan(w[0, 1, :101]).all() and not torch.isnan(w[0, 1, 101:]).any()
    assert torch.equal(w[0, 0], good[0, 0])


def test_hidden_values_do_not_leak_from_few_rows():
    q, k, lse = inputs(1, 30, 400, 4, 2, 128, True, seed=7)
    good = attn_key_weights(q, k, lse)
    bad = k.clone()
    bad[0, 385, 0] = float("nan")
    w = attn_key_weights(q, bad, lse)
    assert torch.isnan(w).nonzero().tolist() == [[0, 0, 385]]
    bad = q.clone()
    bad[0, 10, 3] = float("inf")                    # a row at position 380
    w = attn_key_weights(bad, k, lse)
    assert not torch.isfinite(w[0, 1, :381]).any() and torch.equal(w[0, 1, 381:], good[0, 1, 381:])
    assert torch.equal(w[0, 0], good[0, 0])
    lse[0, 1, 7] = lse[0, 2, 20:] = -float("inf")   # rows without keys
    check(q, k, lse, attn_key_weights(q, k, lse))


@pytest.mark.parametrize("Lq", [400, 30])
def test_a_row_of_nan(Lq):
    """A row whose query and lse are NaN makes the keys that it sees NaN and no others."""
    q, k, lse = inputs(1, Lq, 400, 4, 2, 128, True, seed=12)
    good = attn_key_weights(q, k, lse)
    for row in (0, 13, Lq - 2):
        bad, bad_lse = q.clone(), lse.clone()
        bad[0, row, 2], bad_lse[0, 2, row] = float("nan"), float("nan")
        w = attn_key_weights(bad, k, bad_lse)
        at = 400 - Lq + row
        assert torch.isnan(w[0, 1, :at + 1]).all(), row
        assert torch.equal(w[0, 1, at + 1:], good[0, 1, at + 1:]), row
        assert torch.equal(w[0, 0], good[0, 0]), row


@pytest.mark.parametrize("Lq,n_q,d", [(300, 4, 128), (301, 6, 64), (300, 10, 128), (30, 4, 128), (7, 6, 64)])
def test_a_key_of_weight_zero(Lq, n_q, d):
    """A key whose every score is -inf has weight 0 and changes no other, also where
    a tile has rows that are none (0 * inf)."""
    q, k, lse = inputs(1, Lq, 400, n_q, 2, d, True, seed=Lq)
    q[..., 0] = q[..., 0].abs() + 0.125
    good = attn_key_weights(q, k, lse)
    for j in (37, 390, 399):
        bad = k.clone()
        bad[0, j, :, 0] = -float("inf")
        w = attn_key_weights(q, bad, lse)
        assert (w[..., j] == 0).all(), j
        w[..., j] = good[..., j]
        assert torch.equal(w, good), j


def test_long_prompt_against_the_row_sums():
    """L = 8192 of the 32-head layer: sampled keys in 64 bits, and the total."""
    w = W.WORKLOADS[3]
    q, k, lse = inputs(1, 8192, 8192, 32, 8, 128, True, seed=w.seed)
    got = attn_key_weights(q, k, lse).double()
    assert attn_device_check() == ATTN_OK
    assert abs(got.sum().item() - 32 * 8192) <= 1e-5 * 32 * 8192
    keys = torch.cat([torch.arange(0, 8192, 61), torch.tensor([127, 128, 255, 256, 8190, 8191])]).cuda()
    for u in (0, 3, 7):
        ref = torch.zeros(len(keys), dtype=torch.float64, device="cuda")
        for h in range(4 * u, 4 * u + 4):
            s = q[0, :, h].double() @ k[0, keys, u].double().T * 128 ** -0.5
            p = torch.exp(s - lse[0, h].double()[:, None])
            ref += (p * (keys[None] <= torch.arange(8192, device="cuda")[:, None])).sum(0)
        assert ((got[0, u, keys] - ref).abs() <= 2e-5 * ref).all()


def test_keys_past_2_to_the_31_elements():
    B, Lk, n_kv = 3, 350_000, 24
    k = torch.zeros(B, Lk, n_kv, 128, dtype=torch.bfloat16, device="cuda")
    assert (B - 1) * Lk * n_kv * 128 > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(3)
    for u in (0, n_kv - 1):
        k[2, :, u] = torch.randn(Lk, 128, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(B, 2, 2 * n_kv, 128, generator=g, device="cuda").to(torch.bfloat16)
    lse = torch.full((B, 2 * n_kv, 2), 14.0, device="cuda")
    got = attn_key_weights(q, k, lse).double()
    for u in (0, n_kv - 1):
        ref = torch.zeros(Lk, dtype=torch.float64, device="cuda")
        for h in (2 * u, 2 * u + 1):
            p = torch.exp(k[2, :, u].double() @ q[2, :, h].double().T * 128 ** -0.5 - 14.0)
            p[Lk - 1, 0] = 0
            ref += p.sum(1)
        assert ((got[2, u] - ref).abs() <= 2e-5 * ref).all()
    assert torch.allclose(got[0, 5, :10], torch.full((10,), 4 * np.exp(-14.0), device="cuda",
                                                      dtype=torch.float64), rtol=1e-5)
    del k
    torch.cuda.empty_cache()


def test_graph_streams_and_same_bits():
    q, k, lse = inputs(2, 900, 900, 8, 2, 128, True, seed=8)
    first = attn_key_weights(q, k, lse)
    assert torch.equal(first, attn_key_weights(q, k, lse))
    out = torch.empty_like(first)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn_key_weights(q, k, lse, weights=out, workspace=ws)
    k2 = torch.randn(k.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(9))
    keep = k.clone()
    k.copy_(k2.to(torch.bfloat16))
    other = attn_key_weights(q, k, lse)
    graph.replay()
    assert torch.equal(out, other) and not torch.equal(out, first)
    k.copy_(keep)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [attn_key_weights(q, k, lse, stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(x, first) for x in got)
    assert attn_device_check() == ATTN_OK


def test_refusals():
    q, k, lse = inputs(1, 64, 64, 4, 2, 128, True, seed=1)
    with pytest.raises(ValueError):
        attn_key_weights(q, k[:, :32].contiguous(), lse)
    with pytest.raises(ValueError):
        attn_key_weights(q, k, lse[:, :2].contiguous())
    with pytest.raises(ValueError):
        attn_key_weights(q, k, lse, accumulate=True)
    with pytest.raises(TypeError):
        attn_key_weights(q, k, lse.double())
    with pytest.raises(ValueError):
        attn_key_weights(q.transpose(1, 2), k, lse)
    with pytest.raises(AttnError):
        attn_key_weights(q[..., :32].contiguous(), k[..., :32].contiguous(), lse)
