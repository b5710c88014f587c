"""The cache operators called from several host threads at once, each on a stream of
its own, and a captured call whose rows lose and regain their weight: the bits of the
same calls made alone."""

import threading

import pytest

from cache_common import make
from causal_gqa_prefill_gb300 import (ATTN_OK, attn_decode_ragged, attn_decode_shared,
                                      attn_device_check, attn_evict, attn_key_weights,
                                      attn_key_weights_workspace_bytes, attn_prefill)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def test_threads_at_once():
    g = torch.Generator(device="cuda").manual_seed(70)
    q, k, v, lens, acc = make(6, 2000, 16, 4, [2000, 0, 777, 1, 1999, 128], seed=70, junk=False)
    pk, pv = _normal(g, 1, 1500, 4, 128), _normal(g, 1, 1500, 4, 128)
    ql, kl, vl = _normal(g, 2, 700, 16, 128), _normal(g, 2, 700, 4, 128), _normal(g, 2, 700, 4, 128)
    _, lse = attn_prefill(ql, kl, vl)

    def ragged():
        mine = acc.clone()
        return (*attn_decode_ragged(q, k, v, lens, weights=mine), mine)

    def evict():
        k2, v2, w2, l2, index = attn_evict(k, v, acc, lens, 500, 50)
        past = (torch.arange(500, device="cuda")[None] >= l2[:, None])[..., None, None]
        return k2.masked_fill(past, 0), v2.masked_fill(past, 0), w2, l2, index   # (unspecified there)

    calls = [lambda: (attn_key_weights(ql, kl, lse),),
             lambda: (attn_key_weights(ql[:, -30:].contiguous(), kl, lse[..., -30:].contiguous()),),
             ragged, evict, lambda: attn_decode_shared(q, pk, pv, k, v, lens)]
    alone = [call() for call in calls]
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [calls[i]() for _ in range(20)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:                                           # noqa: BLE001
            errors.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i, want in enumerate(alone):
        for run in got[i]:
            for x, y in zip(run, want):
                assert torch.equal(x, y), i
    assert attn_device_check() == ATTN_OK


@pytest.mark.parametrize("Lq", [600, 40])
def test_graph_follows_padded_rows(Lq):
    """One captured call, replayed while rows lose their weight and get it back."""
    g = torch.Generator(device="cuda").manual_seed(71)
    q, k = _normal(g, 2, Lq, 8, 128), _normal(g, 2, 700, 2, 128)
    _, whole = attn_prefill(q, k, k)
    lse, clean = whole.clone(), q.clone()
    out = torch.empty(2, 2, 700, device="cuda")
    ws = torch.empty(attn_key_weights_workspace_bytes(2, Lq, 700, 8, 2), dtype=torch.uint8,
                     device="cuda")
    good = attn_key_weights(q, k, lse, weights=out, workspace=ws).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn_key_weights(q, k, lse, weights=out, workspace=ws)
    for n in (1, Lq // 2, Lq, 0):
        lse.copy_(whole)
        q.copy_(clean)
        lse[..., Lq - n:] = -float("inf")
        if n:
            q[:, Lq - n:] = float("nan")
        want = attn_key_weights(clean, k, lse)
        graph.replay()
        assert torch.equal(out, want), n
    assert torch.equal(out, good)
    assert attn_device_check() == ATTN_OK
