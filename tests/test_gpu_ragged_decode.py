"""GPU parity of ragged decode against the fp64 oracle, with and without weights.
The tolerances are derived in cache_common.
"""

import pytest

from cache_common import check, make
from causal_gqa_prefill_gb300 import (ATTN_OK, AttnError, attn_decode, attn_decode_ragged,
                                      attn_decode_ragged_workspace_bytes, attn_device_check)

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
    # B, C, n_q, n_kv, lens
    (3, 333, 10, 5, [333, 100, 0]),
    (1, 1, 4, 1, [1]),
    (1, 1, 4, 1, [0]),
    (2, 128, 6, 2, [128, 1]),
    (5, 300, 4, 4, [127, 128, 129, 256, 257]),            # tile edges, g = 1
    (4, 2000, 8, 1, [2000, 1, 1999, 640]),                # g = 8
    (2, 5000, 12, 1, [77, 4999]),                         # g = 12
    (2, 3000, 32, 2, [3000, 1111]),                       # g = 16
    (1, 40000, 36, 6, [39999]),                           # every CTA on one sequence
    (6, 700, 16, 8, [0, 0, 0, 5, 0, 0]),                  # mostly empty
    (3, 50, 8, 2, [0, 0, 0]),                             # all empty
    (40, 260, 14, 2, [(37 * i) % 261 for i in range(40)]),    # runs of sequences per lane, g = 7
    (300, 140, 4, 2, [(53 * i) % 141 for i in range(300)]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_C%d_q%d_kv%d" % c[:4])
@pytest.mark.parametrize("weighted", [False, True])
def test_against_the_oracle(case, weighted):
    q, k, v, lens, acc = make(*case, seed=sum(case[:4]), weights=weighted)
    before = acc.clone() if weighted else None
    o, lse = attn_decode_ragged(q, k, v, lens, weights=acc)
    assert attn_device_check() == ATTN_OK
    check(q, k, v, lens, before, o, lse, acc, what=str(case[:4]))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_other_scales(scale):
    q, k, v, lens, acc = make(2, 500, 8, 2, [500, 123], seed=9)
    before = acc.clone()
    o, lse = attn_decode_ragged(q, k, v, lens, weights=acc, scale=scale)
    check(q, k, v, lens, before, o, lse, acc, scale=scale, what=str(scale))


def test_lengths_out_of_range_are_clamped():
    q, k, v, _, acc = make(2, 200, 8, 2, [200, 200], seed=5)
    lens = torch.tensor([100000, -7], dtype=torch.int32, device="cuda")
    before = acc.clone()
    o, lse = attn_decode_ragged(q, k, v, lens, weights=acc)
    check(q, k, v, lens, before, o, lse, acc)


def test_full_lengths_match_decode():
    q, k, v, lens, _ = make(3, 900, 8, 2, [900] * 3, seed=6, weights=False)
    o, lse = attn_decode_ragged(q, k, v, lens)
    o2, lse2 = attn_decode(q, k, v)
    assert (lse - lse2).abs().max().item() <= 1e-5
    assert (o.float() - o2.float()).abs().max().item() <= 2.0 ** -7 * o2.abs().max().item()


def test_same_bits_again_and_one_workspace():
    ws = torch.full((attn_decode_ragged_workspace_bytes(4, 3000, 8, 2, weighted=True),), 255,
                    dtype=torch.uint8, device="cuda")
    q, k, v, lens, acc = make(4, 3000, 8, 2, [3000, 17, 0, 2222], seed=7)
    runs = []
    for _ in range(3):
        mine = acc.clone()
        o, lse = attn_decode_ragged(q, k, v, lens, weights=mine, workspace=ws)
        runs.append((o, lse, mine))
    torch.cuda.synchronize()
    for o, lse, mine in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])
        assert torch.equal(mine.view(torch.int32), runs[0][2].view(torch.int32))


def test_graph_follows_lengths_and_cache():
    """A captured step replayed while the cache grows, against the same eager steps."""
    B, C, n_q, n_kv = 3, 400, 8, 2
    q, k, v, lens, acc = make(B, C, n_q, n_kv, [127, 0, 260], seed=8, junk=False)
    ws = torch.empty(attn_decode_ragged_workspace_bytes(B, C, n_q, n_kv, weighted=True),
                     dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(B, n_q, 1, device="cuda")
    acc_eager, start = acc.clone(), lens.clone()
    step = lambda w: attn_decode_ragged(q, k, v, lens, weights=w, workspace=ws, out=out, lse=lse)  # noqa: E731
    step(acc.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(acc)
    eager = []
    for _ in range(4):
        step(acc_eager)
        eager.append((out.clone(), lse.clone()))
        lens += 1
    lens.copy_(start)
    for o_e, l_e in eager:
        graph.replay()
        assert torch.equal(out, o_e) and torch.equal(lse, l_e)
        lens += 1
    assert torch.equal(acc, acc_eager)
    assert attn_device_check() == ATTN_OK


def test_two_streams_at_once():
    sets = [make(4, 6000, 8, 2, [6000, 3000 + i, 10, 5999], seed=20 + i) for i in range(2)]
    alone = []
    for q, k, v, lens, acc in sets:
        mine = acc.clone()
        alone.append((*attn_decode_ragged(q, k, v, lens, weights=mine), mine))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    accs = [x[4].clone() for x in sets]
    torch.cuda.synchronize()
    for s, (q, k, v, lens, _), mine in zip(streams, sets, accs):
        got.append((*attn_decode_ragged(q, k, v, lens, weights=mine, stream=s), mine))
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_cache_past_2_to_the_31_elements():
    """The last sequence's rows start 2.15e9 elements into K and V."""
    B, C, n_q, n_kv = 3, 350_000, 48, 24
    k = torch.zeros(B, C, n_kv, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert (B - 1) * C * n_kv * 128 > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    n = 300
    k[2, :n] = torch.randn(n, n_kv, 128, generator=g, device="cuda").to(torch.bfloat16)
    v[2, :n] = torch.randn(n, n_kv, 128, generator=g, device="cuda").to(torch.bfloat16)
    k[2, C - 1], v[2, C - 1] = k[2, 0], v[2, 1]
    q = torch.randn(B, 1, n_q, 128, generator=g, device="cuda").to(torch.bfloat16)
    for last in (n, C):
        lens = torch.tensor([0, 1, last], dtype=torch.int32, device="cuda")
        acc = torch.zeros(B, n_kv, C, device="cuda")
        o, lse = attn_decode_ragged(q, k, v, lens, weights=acc)
        assert attn_device_check() == ATTN_OK
        for u in (0, n_kv - 1):
            qs = q[2, 0, 2 * u:2 * u + 2].double()
            s = qs @ k[2, :last, u].double().T * 128 ** -0.5
            p = torch.softmax(s, 1)
            assert ((p @ v[2, :last, u].double()) - o[2, 0, 2 * u:2 * u + 2].double()).abs().max() < 1e-2
            assert (torch.logsumexp(s, 1) - lse[2, 2 * u:2 * u + 2, 0].double()).abs().max() < 1e-4
            assert torch.allclose(acc[2, u, :last].double(), p.sum(0), rtol=1e-4, atol=0)
    del k, v, acc
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n_q", [2, 8, 24])
def test_a_tile_without_a_finite_score(n_q):
    """Keys whose scores are all -inf have weight 0, also where they are all that a
    tile or a range holds: as if the sequence ended before them."""
    q, k, v, lens, acc = make(2, 700, n_q, 2, [600, 129], seed=11, junk=False)
    q[..., 0] = q[..., 0].abs() + 0.125
    k[0, 256:, :, 0] = k[1, 128:, :, 0] = -float("inf")
    before = acc.clone()
    o, lse = attn_decode_ragged(q, k, v, lens, weights=acc)
    short = torch.tensor([256, 128], dtype=torch.int32, device="cuda")
    check(q, k, v, short, before, o, lse, acc)
    assert attn_device_check() == ATTN_OK


def test_memory_of_another_stream():
    """What a call on another stream allocates is not memory that the current
    stream was given and may still be at work on."""
    q, k, v, lens, acc = make(4, 3000, 8, 2, [3000, 17, 0, 2222], seed=7)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    nbytes = attn_decode_ragged_workspace_bytes(4, 3000, 8, 2)
    mine = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (nbytes, q.nbytes, 512)]
    spans = [(x.untyped_storage().data_ptr(), x.nbytes) for x in mine]
    del mine
    side = torch.cuda.Stream()
    want = attn_decode_ragged(q, k, v, lens)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = attn_decode_ragged(q, k, v, lens, stream=stream)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
            assert all(not at <= x.data_ptr() < at + n for at, n in spans)
    with torch.cuda.stream(side):                  # the default stream by its handle
        got = attn_decode_ragged(q, k, v, lens, stream=0)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_nan_in_visible_places():
    """A NaN query makes its own row NaN and no other; a NaN key those of
    its sequence and K/V head, also where it is all that the sequence has."""
    q, k, v, lens, acc = make(4, 300, 8, 2, [300, 1, 0, 133], seed=3, junk=False)
    good, good_lse = attn_decode_ragged(q, k, v, lens, weights=acc.clone())

    def bad_rows(want, q, k):
        mine = acc.clone()
        o, lse = attn_decode_ragged(q, k, v, lens, weights=mine)
        got = torch.isnan(o[:, 0]).all(2)
        assert got.nonzero().tolist() == want and torch.isnan(o).sum() == 128 * len(want)
        assert torch.equal(torch.isnan(lse[..., 0]), got)
        assert torch.equal(o[:, 0][~got], good[:, 0][~got])
        assert torch.equal(lse[..., 0][~got], good_lse[..., 0][~got])
        heads = got.reshape(4, 2, 4).any(2)
        for b in range(4):
            for u in range(2):
                assert torch.isnan(mine[b, u, :lens[b]]).all() == heads[b, u] or lens[b] == 0
                assert not torch.isnan(mine[b, u, lens[b]:]).any()

    q2, k2 = q.clone(), k.clone()
    q2[0, 0, 3, 7] = q2[1, 0, 5, 0] = float("nan")
    q2[2, 0, 1, 0] = float("nan")                  # a sequence without keys stays 0
    bad_rows([[0, 3], [1, 5]], q2, k)
    k2[1, 0, 1, 9] = k2[3, 130, 0, 9] = float("nan")
    bad_rows([[1, 4], [1, 5], [1, 6], [1, 7], [3, 0], [3, 1], [3, 2], [3, 3]], q, k2)


def test_refusals():
    q, k, v, lens, acc = make(2, 64, 8, 2, [3, 4], seed=1)
    with pytest.raises(ValueError):
        attn_decode_ragged(q, k, v, lens[:1])
    with pytest.raises(TypeError):
        attn_decode_ragged(q, k, v, lens.long())
    with pytest.raises(ValueError):
        attn_decode_ragged(q, k[:, :32], v[:, :32], lens)          # not contiguous
    with pytest.raises(ValueError):
        attn_decode_ragged(q, k, v, lens, weights=acc[:, :1])
    with pytest.raises(ValueError):
        attn_decode_ragged(q.repeat(1, 2, 1, 1), k, v, lens)
    with pytest.raises(AttnError):
        attn_decode_ragged(q, k, v, lens, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(AttnError):
        attn_decode_ragged(q[..., :64].contiguous(), k[..., :64].contiguous(),
                           v[..., :64].contiguous(), lens)
