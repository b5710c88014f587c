"""GPU parity of decode behind a shared prefix against the fp64 oracle. The
tolerances are derived in cache_common."""

import numpy as np
import pytest

from cache_common import check, make
from causal_gqa_prefill_gb300 import (ATTN_OK, AttnError, attn_decode_ragged, attn_decode_shared,
                                      attn_decode_shared_workspace_bytes, attn_device_check)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def inputs(B, P, C, n_q, n_kv, lens, seed, junk=True):
    q, k, v, lens, _ = make(B, C, n_q, n_kv, lens, seed=seed, weights=False, junk=junk)
    g = torch.Generator(device="cuda").manual_seed(seed + 77)
    prefix = [torch.randn(1, P, n_kv, 128, generator=g, device="cuda").to(torch.bfloat16)
              for _ in range(2)]
    return q, prefix, k, v, lens


CASES = [
    # B, P, C, n_q, n_kv, lens
    (1, 1, 1, 1, 1, [0]),
    (1, 1, 1, 4, 1, [1]),
    (2, 127, 40, 8, 2, [40, 0]),
    (4, 1000, 64, 8, 2, [64, 1, 0, 33]),
    (3, 128, 300, 10, 5, [300, 129, 128]),            # one whole prefix tile
    (32, 700, 10, 8, 2, [i % 11 for i in range(32)]),     # exactly one row tile
    (33, 700, 10, 8, 2, [i % 11 for i in range(33)]),     # a second one of four rows
    (64, 1500, 200, 8, 2, [(31 * i) % 201 for i in range(64)]),
    (90, 900, 30, 8, 2, [(7 * i) % 31 for i in range(90)]),   # three row tiles
    (50, 2000, 20, 6, 1, [(3 * i) % 21 for i in range(50)]),  # g = 6: 126 of 128 rows
    (20, 3000, 20, 14, 2, [(3 * i) % 21 for i in range(20)]),  # g = 7
    (130, 400, 9, 2, 2, [i % 10 for i in range(130)]),        # g = 1
    (17, 5000, 50, 32, 2, [(9 * i) % 51 for i in range(17)]),  # g = 16
    (3, 40000, 10, 12, 1, [10, 0, 5]),                        # one unit over every CTA
    (400, 130, 5, 4, 4, [i % 6 for i in range(400)]),         # more units than CTAs' ranges
    (5, 257, 3, 4, 2, [0, 0, 0, 0, 0]),                       # nothing but the prefix
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_P%d_C%d_q%d_kv%d" % c[:5])
def test_against_the_oracle(case):
    q, prefix, k, v, lens = inputs(*case, seed=sum(case[:5]))
    o, lse = attn_decode_shared(q, *prefix, k, v, lens)
    assert attn_device_check() == ATTN_OK
    check(q, k, v, lens, None, o, lse, None, what=str(case[:5]), prefix=prefix)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("B", [5, 70])
def test_other_scales(scale, B):
    q, prefix, k, v, lens = inputs(B, 600, 100, 8, 2, [(13 * i) % 101 for i in range(B)], seed=9)
    o, lse = attn_decode_shared(q, *prefix, k, v, lens, scale=scale)
    check(q, k, v, lens, None, o, lse, None, scale=scale, what=str(scale), prefix=prefix)


@pytest.mark.parametrize("B", [3, 64])
def test_a_prefix_that_peaks_late(B):
    """Scores that grow along the prefix, and own keys far above them: every running
    maximum moves, and one part's weights vanish."""
    q, prefix, k, v, lens = inputs(B, 1000, 60, 8, 2, [(17 * i) % 61 for i in range(B)], seed=10,
                                   junk=False)
    prefix[0] *= torch.linspace(0.1, 12.0, 1000, device="cuda")[None, :, None, None].to(torch.bfloat16)
    k[::2] *= 40
    o, lse = attn_decode_shared(q, *prefix, k, v, lens)
    check(q, k, v, lens, None, o, lse, None, prefix=prefix)


def test_same_as_ragged_decode_over_copies():
    """The same keys, once behind a shared prefix and once copied to every sequence."""
    B, P = 6, 500
    q, prefix, k, v, lens = inputs(B, P, 100, 8, 2, [100, 3, 0, 55, 99, 1], seed=11, junk=False)
    o, lse = attn_decode_shared(q, *prefix, k, v, lens)
    kc, vc = (torch.cat([p.expand(B, -1, -1, -1), x], 1).contiguous()
              for p, x in zip(prefix, (k, v)))
    o2, lse2 = attn_decode_ragged(q, kc, vc, lens + P)
    assert (lse - lse2).abs().max().item() <= 1e-5
    assert (o.float() - o2.float()).abs().max().item() <= 2.0 ** -7 * o2.abs().max().item()


def test_same_bits_again_back_to_back_and_one_workspace():
    """Calls queued on one workspace without a host sync, the caches rewritten by a
    kernel right before each: every call sees its own inputs and partials."""
    B, P, C = 70, 3000, 400
    args = dict(n_q=8, n_kv=2, lens=[(41 * i) % 401 for i in range(B)])
    sets = [inputs(B, P, C, seed=s, junk=False, **args) for s in (21, 22, 23)]
    alone = []
    for q, prefix, k, v, lens in sets:
        alone.append(attn_decode_shared(q, *prefix, k, v, lens))
        torch.cuda.synchronize()
    ws = torch.full((attn_decode_shared_workspace_bytes(B, P, C, 8, 2),), 255, dtype=torch.uint8,
                    device="cuda")
    q0, p0, k0, v0, lens0 = [x.clone() if torch.is_tensor(x) else [y.clone() for y in x]
                             for x in sets[0]]
    got = []
    for q, prefix, k, v, lens in sets * 2:
        for dst, src in zip((q0, *p0, k0, v0), (q, *prefix, k, v)):
            torch.mul(src, 1.0, out=dst)
        got.append(attn_decode_shared(q0, *p0, k0, v0, lens0, workspace=ws))
    torch.cuda.synchronize()
    assert attn_device_check() == ATTN_OK
    for (o, lse), (o1, lse1) in zip(got, alone * 2):
        assert torch.equal(o, o1) and torch.equal(lse, lse1)


def test_graph_follows_lengths_and_cache():
    B, P, C, n_q, n_kv = 40, 700, 50, 8, 2
    q, prefix, k, v, lens = inputs(B, P, C, n_q, n_kv, [i % 40 for i in range(B)], seed=8, junk=False)
    ws = torch.empty(attn_decode_shared_workspace_bytes(B, P, C, n_q, n_kv), dtype=torch.uint8,
                     device="cuda")
    out, lse = torch.empty_like(q), torch.empty(B, n_q, 1, device="cuda")
    step = lambda: attn_decode_shared(q, *prefix, k, v, lens, workspace=ws, out=out, lse=lse)  # noqa: E731
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    start, eager = lens.clone(), []
    for _ in range(3):
        step()
        eager.append((out.clone(), lse.clone()))
        lens += 3
    lens.copy_(start)
    for o_e, l_e in eager:
        graph.replay()
        assert torch.equal(out, o_e) and torch.equal(lse, l_e)
        lens += 3
    assert attn_device_check() == ATTN_OK


def test_two_streams_at_once():
    sets = [inputs(40, 3000, 300, 8, 2, [(11 * i) % 301 for i in range(40)], seed=s) for s in (31, 32)]
    alone = [attn_decode_shared(q, *p, k, v, lens) for q, p, k, v, lens in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(3):
        got += [attn_decode_shared(q, *p, k, v, lens, stream=s)
                for s, (q, p, k, v, lens) in zip(streams, sets)]
    torch.cuda.synchronize()
    for (o, lse), (o1, lse1) in zip(got, alone * 3):
        assert torch.equal(o, o1) and torch.equal(lse, lse1)


def test_large_batch_on_sampled_rows():
    """256 sequences of the 64-head layer behind 32768 positions, sampled heads in 64 bits."""
    B, P, C, n_q, n_kv = 256, 32768, 128, 64, 8
    rng = np.random.default_rng(3)
    q, prefix, k, v, lens = inputs(B, P, C, n_q, n_kv, rng.integers(0, C + 1, B).tolist(), seed=40)
    o, lse = attn_decode_shared(q, *prefix, k, v, lens)
    assert attn_device_check() == ATTN_OK
    for b, h in [(0, 0), (255, 63), (15, 7), (16, 8), (127, 31), (200, 40), (31, 56)]:
        n = int(lens[b])
        ks, vs = (torch.cat([p[0, :, h // 8], x[b, :n, h // 8]]).double()
                  for p, x in zip(prefix, (k, v)))
        s = ks @ q[b, 0, h].double() * 128 ** -0.5
        p = torch.softmax(s, 0)
        ref, size = p @ vs, p @ vs.abs()
        err = (o[b, 0, h].double() - ref).abs()
        assert (err <= 2.0 ** -8 * ((1 + 2.0 ** -6) * size + ref.abs())).all(), (b, h)
        assert abs(torch.logsumexp(s, 0) - lse[b, h, 0].double()) <= 1e-4


def test_nan_in_visible_places():
    """A NaN query makes its own row NaN and no other; a NaN key those of
    its sequence and K/V head, also where it is all that the sequence has."""
    q, prefix, k, v, lens = inputs(4, 300, 40, 8, 2, [40, 1, 0, 33], seed=3, junk=False)
    good, good_lse = attn_decode_shared(q, *prefix, k, v, lens)

    def bad_rows(want, *args):
        o, lse = attn_decode_shared(*args, lens)
        got = torch.isnan(o[:, 0]).all(2)
        assert got.nonzero().tolist() == want and torch.isnan(o).sum() == 128 * len(want)
        assert torch.equal(torch.isnan(lse[..., 0]), got)
        assert torch.equal(o[:, 0][~got], good[:, 0][~got])
        assert torch.equal(lse[..., 0][~got], good_lse[..., 0][~got])

    q2, k2, p2 = q.clone(), k.clone(), prefix[0].clone()
    q2[0, 0, 3, 7] = q2[2, 0, 5, 0] = float("nan")
    bad_rows([[0, 3], [2, 5]], q2, *prefix, k, v)
    k2[1, 0, 1, 9] = float("nan")                  # the only own position of sequence 1
    k2[3, 20, 0, 9] = float("nan")
    bad_rows([[1, 4], [1, 5], [1, 6], [1, 7], [3, 0], [3, 1], [3, 2], [3, 3]], q, *prefix, k2, v)
    p2[0, 299, 1, 0] = float("nan")
    bad_rows([[b, h] for b in range(4) for h in range(4, 8)], q, p2, prefix[1], k, v)


def test_refusals():
    q, prefix, k, v, lens = inputs(2, 64, 32, 8, 2, [3, 4], seed=1)
    with pytest.raises(ValueError):
        attn_decode_shared(q, prefix[0][0], prefix[1][0], k, v, lens)
    with pytest.raises(ValueError):
        attn_decode_shared(q, prefix[0], prefix[1][:, :32].contiguous(), k, v, lens)
    with pytest.raises(ValueError):
        attn_decode_shared(q, *prefix, k[:1], v[:1], lens)
    with pytest.raises(TypeError):
        attn_decode_shared(q, *prefix, k, v, lens.long())
    with pytest.raises(AttnError):
        attn_decode_shared(q, *prefix, k, v, lens,
                           workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
