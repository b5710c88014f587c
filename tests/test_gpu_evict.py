"""GPU parity of cache eviction with the oracle: index, lengths, weights and rows
are equal, bit by bit."""

import numpy as np
import pytest

import oracle
from causal_gqa_prefill_gb300 import ATTN_OK, AttnError, attn_device_check, attn_evict

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def rows(shape, dtype, g):
    """Rows of random bytes: a copy is a copy whatever they stand for."""
    size = torch.empty((), dtype=dtype).element_size()
    x = torch.randint(0, 256, (*shape[:-1], shape[-1] * size), generator=g, device="cuda",
                      dtype=torch.uint8)
    return x.view(dtype)


def make(B, C, n_kv, d, dtype, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = rows((B, C, n_kv, d), dtype, g), rows((B, C, n_kv, d), dtype, g)
    w = torch.rand(B, n_kv, C, generator=g, device="cuda")
    if kind == "ties":                                    # seven values, one of them -0
        w = (w * 7).floor() / 7
        w = torch.where(w == 0, -w, w)
        w[..., ::3] = w[..., ::3].abs()
    elif kind == "wild":                                  # signs, infinities, NaN, subnormals
        w = torch.randn(B, n_kv, C, generator=g, device="cuda") * 1e3
        pick = torch.randint(0, 8, w.shape, generator=g, device="cuda")
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), 1e-41, -1e-41)):
            w[pick == i] = x
    elif kind == "equal":
        w = torch.ones_like(w)
    return k, v, w


def check(k, v, w, lens, budget, recent, capacity=None, **kw):
    B, C, n_kv, d = k.shape
    cap = capacity or budget
    fill = {"k_out": rows((B, cap, n_kv, d), k.dtype, torch.Generator(device="cuda").manual_seed(9)),
            "v_out": rows((B, cap, n_kv, d), k.dtype, torch.Generator(device="cuda").manual_seed(8))}
    old = {n: t.clone() for n, t in fill.items()}
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k2, v2, w2, l2, index = attn_evict(k, v, w, lens, budget, recent, capacity=capacity, **fill, **kw)
    assert attn_device_check() == ATTN_OK
    ref, new = oracle.cache.evicted_index(w.cpu().numpy(), lens.cpu().numpy(), budget, recent)
    assert np.array_equal(l2.cpu().numpy(), new)
    assert np.array_equal(index.cpu().numpy(), ref)
    at = torch.from_numpy(ref.astype(np.int64)).cuda()
    live = at >= 0
    w_ref = torch.zeros(B, n_kv, cap, device="cuda")
    w_ref[..., :budget] = torch.where(live, w.gather(2, at.clamp(min=0)), 0.0)
    assert torch.equal(w_ref.view(torch.int32), w2.view(torch.int32))
    for src, dst, was in ((k, k2, old["k_out"]), (v, v2, old["v_out"])):
        src, dst, was = (x.view(torch.uint8) for x in (src, dst, was))
        pos = at.clamp(min=0).transpose(1, 2)[..., None].expand(-1, -1, -1, src.shape[-1])
        want = was.clone()
        want[:, :budget] = torch.where(live.transpose(1, 2)[..., None], src.gather(1, pos),
                                       was[:, :budget])
        assert torch.equal(dst, want)


CASES = [
    # B, C, n_kv, lens, budget, recent, capacity
    (1, 1, 1, [1], 1, 0, None),
    (2, 8, 1, [8, 3], 4, 1, None),
    (3, 333, 5, [333, 100, 0], 100, 7, 130),
    (2, 500, 2, [500, 77], 1, 1, None),                 # one position, the last
    (2, 500, 2, [500, 499], 64, 64, None),              # only recent ones
    (2, 500, 2, [500, 499], 499, 0, 500),               # all but one
    (2, 500, 3, [500, 200], 500, 10, 600),              # nothing to evict
    (4, 2049, 2, [2049, 2048, 1025, 1023], 1024, 100, None),
    (1, 9000, 2, [9000], 4000, 10, None),               # a cluster of two
    (2, 20000, 3, [20000, 19999], 5000, 1000, None),    # of four
    (1, 70001, 2, [70001], 7000, 0, 8000),              # of eight
    (1, 70001, 2, [9], 7000, 0, None),                  # of eight, almost nothing there
    (50, 129, 4, [(17 * i) % 130 for i in range(50)], 60, 20, 64),
]


@pytest.mark.parametrize("kind", ["plain", "ties", "wild", "equal"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_C%d_kv%d_%s" % (c[0], c[1], c[2], c[4]))
def test_against_the_oracle(case, kind):
    B, C, n_kv, lens, budget, recent, capacity = case
    i = CASES.index(case)
    d, dtype = ((128, torch.bfloat16), (64, torch.bfloat16), (128, torch.float8_e4m3fn),
                (64, torch.float8_e4m3fn))[i % 4]
    check(*make(B, C, n_kv, d, dtype, kind, seed=i), lens, budget, recent, capacity)


@pytest.mark.parametrize("B,C,n_kv", [(160, 41100, 1), (1, 330000, 1)])
def test_parts_too_long_for_shared_memory(B, C, n_kv):
    k, v, w = make(B, C, n_kv, 64, torch.float8_e4m3fn, "plain", seed=3)
    check(k, v, w, [C - 3 * i for i in range(B)], 500, 20)


@pytest.mark.parametrize("C,near", [(20000, 3), (70001, 40), (70001, 127), (330000, 100), (500, 128)])
def test_the_last_few_are_near_or_equal(C, near):
    """Most weights far apart, and as many as are listed and compared one by one (or
    one more) that differ in their last bits or not at all, spread over all CTAs."""
    k, v, w = make(1, C, 2, 64, torch.float8_e4m3fn, "plain", seed=C + near)
    g = torch.Generator().manual_seed(near)
    for extra in (0, 2):
        at = torch.randperm(C - 20, generator=g)[:near + extra].cuda()
        bits = torch.full((near + extra,), 0x3F812300, dtype=torch.int32, device="cuda")
        w.copy_(torch.rand(w.shape, device="cuda") * 0.9 + 4.0 * (torch.rand(w.shape, device="cuda") < 0.01))
        bits += torch.randint(0, 4, bits.shape, generator=g, dtype=torch.int32).cuda()
        w[0, 0, at] = bits.view(torch.float32)
        w[0, 1, at] = 1.0087890625
        larger = int((w[0, :, :C - 20] >= 2).sum(1).max())
        for n in (1, near // 2 + 1, near):
            check(k, v, w, [C], 20 + larger + n, 20)


def test_lengths_out_of_range_are_clamped():
    k, v, w = make(2, 100, 2, 64, torch.bfloat16, "plain", seed=4)
    check(k, v, w, [1000, -5], 30, 5)


def test_source_past_2_to_the_31_elements():
    B, C, n_kv, d = 3, 350_000, 24, 128
    k = torch.zeros(B, C, n_kv, d, dtype=torch.bfloat16, device="cuda")
    assert (B - 1) * C * n_kv * d > 2 ** 31
    v = torch.zeros_like(k)
    k[..., 0] = (torch.arange(C, device="cuda") % 251).to(torch.bfloat16)[None, :, None]
    v[..., 1] = (torch.arange(C, device="cuda") % 241).to(torch.bfloat16)[None, :, None]
    w = torch.rand(B, n_kv, C, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    lens = torch.full((B,), C, dtype=torch.int32, device="cuda")
    k2, v2, w2, l2, index = attn_evict(k, v, w, lens, 2000, 100)
    order = w[..., :C - 100].sort(dim=-1, descending=True, stable=True)[1]
    top = order[..., :1900].sort(-1)[0]
    assert torch.equal(index[..., :1900].long(), top)
    assert torch.equal(k2[..., 0].transpose(1, 2).float(), (index % 251).float())
    assert torch.equal(v2[..., 1].transpose(1, 2).float(), (index % 241).float())
    del k, v, k2, v2
    torch.cuda.empty_cache()


def test_graph_replay_follows_its_inputs():
    k, v, w = make(2, 5000, 2, 128, torch.bfloat16, "plain", seed=5)
    lens = torch.tensor([5000, 3000], dtype=torch.int32, device="cuda")
    outs = dict(zip(("k_out", "v_out", "weights_out", "lens_out", "index"),
                    attn_evict(k, v, w, lens, 700, 30, capacity=800)))
    outs["k_out"].zero_(), outs["v_out"].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn_evict(k, v, w, lens, 700, 30, **outs)
    w.copy_(torch.rand(w.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(6)))
    lens.copy_(torch.tensor([600, 4999], dtype=torch.int32))
    graph.replay()
    got = {n: t.clone() for n, t in outs.items()}
    outs["k_out"].zero_(), outs["v_out"].zero_()
    attn_evict(k, v, w, lens, 700, 30, **outs)
    torch.cuda.synchronize()
    for n, t in outs.items():
        same = torch.equal if t.dtype != torch.bfloat16 else \
            (lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16)))
        assert same(t, got[n]), n


def test_two_streams_at_once():
    sets = [make(4, 9000, 2, 128, torch.bfloat16, "ties", seed=30 + i) for i in range(2)]
    lens = torch.tensor([9000, 8000, 100, 4097], dtype=torch.int32, device="cuda")
    alone = [attn_evict(*x, lens, 3000, 100)[2:] for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [attn_evict(*x, lens, 3000, 100, stream=s)[2:] for x, s in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_refusals():
    k, v, w = make(2, 100, 2, 64, torch.bfloat16, "plain", seed=7)
    lens = torch.tensor([100, 50], dtype=torch.int32, device="cuda")
    for bad in (0, -1):
        with pytest.raises(ValueError):
            attn_evict(k, v, w, lens, bad)
    with pytest.raises(ValueError):
        attn_evict(k, v, w, lens, 10, 11)
    with pytest.raises(ValueError):
        attn_evict(k, v, w, lens, 10, capacity=9)
    with pytest.raises(ValueError):
        attn_evict(k, v, w[:, :1], lens, 10)
    with pytest.raises(TypeError):
        attn_evict(k, v, w.double(), lens, 10)
    with pytest.raises(AttnError):                       # in place
        attn_evict(k, v, w, lens, 10, k_out=k, capacity=100)
    with pytest.raises(AttnError):
        attn_evict(k, v, w, lens, 10, lens_out=lens)
    with pytest.raises(AttnError):
        attn_evict(k[..., :32].contiguous(), v[..., :32].contiguous(), w, lens, 10)
