"""The cache operators as a program uses them, one after another: prefill, the
weights of its keys, eviction to a budget, decode steps that append and go on
weighing, eviction again; a prefix kept once and shared by the answers to it.
Every call is checked against the oracle on what the call before it left."""

import json
import os
import subprocess
import sys

import numpy as np
import pytest

import oracle
from cache_common import check
from causal_gqa_prefill_gb300 import (ATTN_ERR_UNSUPPORTED, ATTN_OK, attn_decode_ragged,
                                      attn_decode_ragged_workspace_bytes, attn_decode_shared,
                                      attn_device_check, attn_evict, attn_key_weights, attn_prefill)
from gpu_common import check_full, to_np

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def test_prefill_weights_evict_decode():
    B, L, n_q, n_kv, budget, recent, room = 2, 700, 8, 2, 150, 20, 160
    g = torch.Generator(device="cuda").manual_seed(60)
    q, k, v = _normal(g, B, L, n_q, 128), _normal(g, B, L, n_kv, 128), _normal(g, B, L, n_kv, 128)
    o, lse = attn_prefill(q, k, v)
    check_full(q, k, v, o, lse)

    weights = attn_key_weights(q, k, lse)
    ref = oracle.cache.key_weights(to_np(q), to_np(k), lse.cpu().numpy().astype(np.float64))
    assert np.allclose(weights.cpu().numpy(), ref, rtol=1e-4, atol=0)

    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    k, v, weights, lens, index = attn_evict(k, v, weights, lens, budget, recent, capacity=room)
    kept, _ = oracle.cache.evicted_index(ref, [L] * B, budget, recent)
    # (the oracle's weights and the kernel's may order near-equal ones differently)
    assert (index.cpu().numpy() == kept).mean() > 0.99
    assert lens.tolist() == [budget] * B

    ws = torch.empty(attn_decode_ragged_workspace_bytes(B, room, n_q, n_kv, weighted=True),
                     dtype=torch.uint8, device="cuda")
    rows = torch.arange(B, device="cuda")
    for step in range(25):                                  # room for 10 between evictions
        if int(lens.max()) == room:
            before = weights.cpu().numpy(), lens.cpu().numpy()
            k, v, weights, lens, index = attn_evict(k, v, weights, lens, budget, recent, capacity=room)
            kept, new = oracle.cache.evicted_index(*before, budget, recent)
            assert np.array_equal(index.cpu().numpy(), kept) and np.array_equal(lens.cpu().numpy(), new)
            assert (weights[..., budget:] == 0).all()
        at = lens.long()
        k[rows, at], v[rows, at] = _normal(g, B, n_kv, 128), _normal(g, B, n_kv, 128)
        lens += 1
        qs, was = _normal(g, B, 1, n_q, 128), weights.clone()
        o, lse = attn_decode_ragged(qs, k, v, lens, weights=weights, workspace=ws)
        check(qs, k, v, lens, was, o, lse, weights, what=f"step {step}")
    assert attn_device_check() == ATTN_OK


def test_one_prompt_many_answers():
    """A prompt prefilled once, its K and V used as the shared prefix of a batch
    whose answers grow, the whole step in one captured graph."""
    L, B, room, n_q, n_kv = 300, 20, 40, 8, 2
    g = torch.Generator(device="cuda").manual_seed(61)
    q, pk, pv = _normal(g, 1, L, n_q, 128), _normal(g, 1, L, n_kv, 128), _normal(g, 1, L, n_kv, 128)
    check_full(q, pk, pv, *attn_prefill(q, pk, pv))
    k, v = (torch.zeros(B, room, n_kv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    rows = torch.arange(B, device="cuda")
    new_q, new_k, new_v = (_normal(g, B, 1, n_q, 128), _normal(g, B, n_kv, 128),
                           _normal(g, B, n_kv, 128))

    def step():
        at = lens.long()
        k[rows, at] = new_k
        v[rows, at] = new_v
        lens.add_(1)
        return attn_decode_shared(new_q, pk, pv, k, v, lens)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    for _ in range(5):
        new_q.copy_(_normal(g, B, 1, n_q, 128))
        new_k.copy_(_normal(g, B, n_kv, 128))
        new_v.copy_(_normal(g, B, n_kv, 128))
        graph.replay()
        torch.cuda.synchronize()
        check(new_q, k, v, lens, None, o, lse, None, prefix=(pk, pv))
    assert lens.tolist() == [6] * B
    assert attn_device_check() == ATTN_OK


_FIRST_CALL = r"""
import json, torch
import causal_gqa_prefill_gb300 as cg
torch.cuda.set_device(0)
q = torch.randn(2, 1, 4, 128, device="cuda").to(torch.bfloat16)
k = torch.randn(2, 256, 2, 128, device="cuda").to(torch.bfloat16)
v, p = torch.randn_like(k), torch.randn_like(k[:1])
lens = torch.tensor([256, 100], dtype=torch.int32, device="cuda")
w = torch.rand(2, 2, 256, device="cuda")
lse = torch.zeros(2, 4, 1, device="cuda")
torch.cuda.synchronize()
calls = {"weights": lambda: cg.attn_key_weights(q, k, lse),
         "evict": lambda: cg.attn_evict(k, v, w, lens, 50, 10),
         "shared": lambda: cg.attn_decode_shared(q, p, p, k, v, lens),
         "ragged": lambda: cg.attn_decode_ragged(q, k, v, lens, weights=w)}
res = {}
for name in ORDER:
    try:
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            calls[name]()
        res[name + "_capture"] = "ok"
    except cg.AttnError as e:
        res[name + "_capture"] = e.status
    calls[name]()
    torch.cuda.synchronize()
    res[name + "_eager"] = cg.attn_device_check()
print(json.dumps(res))
"""


@pytest.mark.parametrize("order", [["weights", "evict", "shared"], ["ragged"]])
def test_first_call_during_capture_is_refused(order):
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALL.replace("ORDER", repr(order))], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    for name in order:
        assert res[name + "_capture"] == ATTN_ERR_UNSUPPORTED, res
        assert res[name + "_eager"] == ATTN_OK, res
