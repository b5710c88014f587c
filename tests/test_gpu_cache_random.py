"""A seeded sweep of random small shapes of the cache operators against the fp64
oracle, every element: any group size, lengths at tile edges and anywhere, d_h 64
and 128, chunks anywhere in a prompt, causal and full, other scales. The tolerances
are those of the operators' own tests.
"""

import random

import pytest

import cache_common
import test_gpu_evict as evict
import test_gpu_key_weights as weights
from causal_gqa_prefill_gb300 import (ATTN_OK, attn_decode_ragged, attn_decode_shared,
                                      attn_device_check, attn_key_weights)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def length(rng, most):
    """Often at a tile's edge, else anywhere."""
    if rng.random() < 0.5:
        return max(1, min(most, rng.choice([1, 2, 64, 128, 256, 384, 512, 640]) + rng.randint(-1, 1)))
    return rng.randint(1, most)


def lens_of(rng, B, C):
    return [rng.choice([0, C, length(rng, C), rng.randint(0, C)]) for _ in range(B)]


@pytest.mark.parametrize("seed", range(40))
def test_key_weights(seed):
    rng = random.Random(seed)
    n_kv, g, d = rng.randint(1, 3), rng.choice([1, 2, 3, 4, 5, 6, 8, 9, 16, 31, 64, 128]), rng.choice([64, 128])
    B, Lk = rng.randint(1, 3), length(rng, 700)
    Lq = rng.choice([Lk, length(rng, Lk), rng.randint(1, Lk)])
    Lq = max(1, min(Lq, Lk, 40000 // (g * n_kv * B)))
    causal, scale = rng.random() < 0.7, rng.choice([None, None, -0.1, 0.3])
    q, k, lse = weights.inputs(B, Lq, Lk, g * n_kv, n_kv, d, causal, seed, scale=scale)
    before = torch.rand(B, n_kv, Lk, device="cuda") if rng.random() < 0.4 else None
    got = None if before is None else before.clone()
    got = attn_key_weights(q, k, lse, causal=causal, scale=scale, weights=got,
                           accumulate=before is not None)
    assert attn_device_check() == ATTN_OK
    weights.check(q, k, lse, got, causal, scale, before, what=str((B, Lq, Lk, g, n_kv, d, causal)))


@pytest.mark.parametrize("seed", range(40))
def test_ragged_decode(seed):
    rng = random.Random(1000 + seed)
    B, C, n_kv, g = rng.randint(1, 9), length(rng, 900), rng.randint(1, 6), rng.randint(1, 16)
    weighted, scale = rng.random() < 0.6, rng.choice([None, None, -0.1, 0.3])
    q, k, v, lens, acc = cache_common.make(B, C, g * n_kv, n_kv, lens_of(rng, B, C), seed=seed,
                                           weights=weighted)
    before = acc.clone() if weighted else None
    o, lse = attn_decode_ragged(q, k, v, lens, weights=acc, scale=scale)
    assert attn_device_check() == ATTN_OK
    cache_common.check(q, k, v, lens, before, o, lse, acc, scale=scale, what=str((B, C, g, n_kv)))


@pytest.mark.parametrize("seed", range(40))
def test_shared_prefix(seed):
    rng = random.Random(2000 + seed)
    B, C, n_kv, g = rng.randint(1, 70), length(rng, 400), rng.randint(1, 3), rng.randint(1, 16)
    P, scale = length(rng, 1500), rng.choice([None, None, -0.1, 0.3])
    q, k, v, lens, _ = cache_common.make(B, C, g * n_kv, n_kv, lens_of(rng, B, C), seed=seed,
                                         weights=False)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pk, pv = (torch.randn(1, P, n_kv, 128, generator=gen, device="cuda").to(torch.bfloat16)
              for _ in range(2))
    o, lse = attn_decode_shared(q, pk, pv, k, v, lens, scale=scale)
    assert attn_device_check() == ATTN_OK
    cache_common.check(q, k, v, lens, None, o, lse, None, scale=scale, what=str((B, P, C, g, n_kv)),
                       prefix=(pk, pv))


@pytest.mark.parametrize("seed", range(40))
def test_evict(seed):
    rng = random.Random(3000 + seed)
    B, C, n_kv = rng.randint(1, 20), rng.choice([length(rng, 700), rng.randint(1, 20000)]), rng.randint(1, 4)
    budget = rng.choice([1, C, C + 7, rng.randint(1, C), rng.randint(1, C)])
    recent = rng.choice([0, budget, rng.randint(0, budget)])
    capacity = budget + rng.choice([0, 0, 1, 77])
    d, dtype = rng.choice([64, 128]), rng.choice([torch.bfloat16, torch.float8_e4m3fn])
    kind = rng.choice(["plain", "plain", "ties", "wild", "equal"])
    evict.check(*evict.make(B, C, n_kv, d, dtype, kind, seed=seed), lens_of(rng, B, C), budget, recent,
                capacity)
