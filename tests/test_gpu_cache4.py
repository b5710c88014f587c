"""GPU parity of caches held in 4 bits: packing and unpacking bit for bit, decode
against the fp64 reference on the values that the codes stand for.

Tolerance of decode. A score is an fp32 sum over groups of scale_g sum (16 + code) q
and (lo_g - 16 scale_g) sum q: with every magnitude added up, S_abs = scale sum_g
sum|q| (47 scale_g + |lo_g|), some six roundings of 2^-23 make E = 2^-20 S_abs. LSE
is off by E + 2^-20 + 2^-22 |LSE|. O: bf16 (p scale_g) times the codes less c is off
by 2^-8 A, A = sum p |V - mid|, mid = lo + scale c, c the nearest of 0 .. 15 to
-lo / scale (to within 15 2^-22, three fp32 roundings: where two are that near, either,
a scale further off); the fp32 parts (scores, exponentials, sum p mid) by (2 E + 2^-20)
(sum p (|lo| + |V|) + |O|), where |mid| <= |V| + |V - mid|; 2^-6 A 2^-8 covers both on
A; O rounds once: 2^-8 |O|.
"""

import numpy as np
import pytest

from causal_gqa_prefill_gb300 import (ATTN_OK, AttnError, attn_decode4, attn_decode4_workspace_bytes,
                                      attn_device_check, attn_pack4, attn_unpack4)
from causal_gqa_prefill_gb300 import workloads as W
from gpu_common import to_np
from oracle import cache4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from causal_gqa_prefill_gb300 import build
    build.build()
    torch.cuda.set_device(0)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(B, L, n_kv, seed=0, kind="normal"):
    """bf16 rows [B, L, n_kv, 128], of values where a code is hard to tell."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((B, L, n_kv, 128))
    if kind == "outliers":
        x[..., 5::32] *= 50
    elif kind == "grid":                 # many quotients on a border
        x = rng.integers(-60, 61, x.shape) * 0.25
        x[..., ::32], x[..., 1::32] = -15.0, 15.0
    elif kind == "spread":               # exponents far apart: differences that fp32 rounds
        x = x * 2.0 ** rng.integers(-40, 5, x.shape)
        x[..., 2::32] = rng.choice([1.0, 3.5, 7.5, 0.46875], x[..., 2::32].shape)
        x[..., 3::32] = -x[..., 2::32]
    elif kind == "tiny":
        x = x * 2.0 ** rng.integers(-135, -115, x.shape[:-1] + (1,))
    elif kind == "huge":
        x = np.clip(x * 1.5e38, -3.38e38, 3.38e38)
    elif kind == "odd":
        x[rng.random(x.shape) < 0.004] = np.nan
        x[rng.random(x.shape) < 0.004] = np.inf
        x[rng.random(x.shape) < 0.004] = -np.inf
    elif kind == "flat":
        x = np.broadcast_to(x[..., :1], x.shape)
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).cuda()


def stored(cache, x, at, counts=None):
    """What the reference makes of the caches [B, n_kv, C, 80]."""
    out = cache.cpu().numpy().copy()
    packed = cache4.pack(x.double().cpu().numpy())
    for b in range(x.shape[0]):
        for i in range(x.shape[1] if counts is None else min(counts[b], x.shape[1])):
            pos = at[b] + i
            if 0 <= pos < out.shape[2]:
                out[b, :, pos] = packed[b, i]
    return out


def read(cache, at, L):
    """What unpacking gives: bf16 [B, L, n_kv, 128] as float64."""
    B, n_kv, C, _ = cache.shape
    val = cache4.rounded(cache)
    out = np.zeros((B, L, n_kv, 128))
    for b in range(B):
        for i in range(L):
            if 0 <= at[b] + i < C:
                out[b, i] = val[b, :, at[b] + i]
    return out


CASES = [
    # B, L, C, n_kv, at, counts
    (1, 1, 1, 1, [0], None),
    (2, 5, 9, 3, [4, 0], None),
    (3, 7, 20, 2, [0, 13, 5], [7, 0, 3]),
    (2, 6, 8, 1, [5, -3], None),                     # rows past either end are left out
    (2, 3, 8, 2, [100, -100], None),
    (2, 4, 8, 2, [1, 2], [99, -5]),
    (64, 1, 40, 8, [(7 * b) % 40 for b in range(64)], None),
    (1, 300, 333, 5, [33], None),
    (3, 129, 140, 1, [11, 3, 0], [129, 64, 1]),
]


@pytest.mark.parametrize("kind", ["normal", "outliers", "grid", "spread", "tiny", "huge", "odd", "flat"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_L%d_C%d_kv%d" % c[:4])
def test_rows_bit_for_bit(case, kind):
    B, L, C, n_kv, at, counts = case
    k, v = rows(B, L, n_kv, 1, kind), rows(B, L, n_kv, 2, kind)
    k4, v4 = (torch.randint(0, 256, (B, n_kv, C, 80), dtype=torch.uint8, device="cuda")
              for _ in range(2))
    want = [stored(c, x, at, counts) for c, x in ((k4, k), (v4, v))]
    attn_pack4(k, v, k4, v4, i32(*at), counts=None if counts is None else i32(*counts))
    for c, ref in zip((k4, v4), want):
        assert np.array_equal(c.cpu().numpy(), ref)
    k2, v2 = attn_unpack4(k4, v4, L, i32(*at))
    assert attn_device_check() == ATTN_OK
    for x, ref in zip((k2, v2), want):
        ref = read(ref, at, L)
        x = x.double().cpu().numpy()
        # lo + scale code, rounded once
        assert ((x == ref) | (np.isnan(x) & np.isnan(ref))).all()


def test_rows_without_positions_begin_at_zero():
    k, v = rows(2, 9, 2, 3), rows(2, 9, 2, 4)
    a, b = (torch.zeros(2, 2, 12, 80, dtype=torch.uint8, device="cuda") for _ in range(2))
    attn_pack4(k, v, a, b)
    assert np.array_equal(a.cpu().numpy(), stored(torch.zeros_like(a), k, [0, 0]))
    assert not a[:, :, 9:].any() and not b[:, :, 9:].any()
    k2, v2 = attn_unpack4(a, b, 5)
    assert torch.equal(k2, attn_unpack4(a, b, 12)[0][:, :5])
    # read again, packed again: lo and the codes of what 4 bits hold
    c, d = (torch.zeros(2, 2, 5, 80, dtype=torch.uint8, device="cuda") for _ in range(2))
    attn_pack4(k2, v2, c, d)
    k3, _ = attn_unpack4(c, d, 5)
    assert (k3.float() - k2.float()).abs().max() <= 0.05 * k2.abs().max()


def test_a_cache_past_32_bits():
    """Positions whose bytes lie beyond 2^31 and 2^32."""
    C, n_kv = 1 << 25, 2
    k4 = torch.zeros(1, n_kv, C, 80, dtype=torch.uint8, device="cuda")
    v4 = torch.zeros_like(k4)
    k, v = rows(1, 700, n_kv, 5), rows(1, 700, n_kv, 6)
    at = C - 700
    attn_pack4(k, v, k4, v4, i32(at))
    assert np.array_equal(k4[:, :, at:].cpu().numpy(), stored(torch.zeros(1, n_kv, 700, 80), k, [0])
                          .astype(np.uint8))
    k2, v2 = attn_unpack4(k4, v4, 700, i32(at))
    assert torch.equal(v2, attn_unpack4(v4[:, :, at:].contiguous(), v4[:, :, at:].contiguous(), 700)[0])
    q = W.make_inputs(W.custom(1, 1, 4, n_kv, 128, Lk=4), "cuda", seed=7)[0]
    o, lse = attn_decode4(q, k4, v4, i32(C), window=600)
    check_step(q, k4[:, :, -600:], v4[:, :, -600:], [600], o, lse, None, 0)


# -------------------------------------------------------------------- decode


def check_step(q, k4, v4, lens, o, lse, window, sinks, scale=None, what=""):
    q, o, lse = to_np(q), to_np(o), lse.cpu().numpy().astype(np.float64)
    B, _, n_q, d = q.shape
    n_kv, C = k4.shape[1:3]
    g, scale = n_q // n_kv, d ** -0.5 if scale is None else scale
    for b in range(B):
        n = min(max(lens[b], 0), C)
        if n == 0:
            assert not o[b].any() and (lse[b] == -np.inf).all(), what
            continue
        first = max(0, n - window) if window else 0
        at = [*range(min(sinks, first)), *range(first, n)]
        for u in range(n_kv):
            K, klo = cache4.unpack(k4[b, u, at].cpu().numpy())
            V, vlo = cache4.unpack(v4[b, u, at].cpu().numpy())
            bits = k4[b, u, at].cpu().numpy()
            step = np.repeat(cache4.bf16_value(bits[:, 64::4].astype(np.uint32)
                                               | bits[:, 65::4].astype(np.uint32) << 8), 32, axis=1)
            Q = q[b, 0, u * g:u * g + g]
            s = scale * (Q @ K.T)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(1, keepdims=True)
            p /= total
            ref, ref_lse = p @ V, (m + np.log(total))[:, 0]
            E = 2.0 ** -20 * abs(scale) * (np.abs(Q) @ (47 * step + np.abs(klo)).T).max(1)
            off = np.abs(lse[b, u * g:u * g + g, 0] - ref_lse)
            assert (off <= E + 2.0 ** -20 + 2.0 ** -22 * np.abs(ref_lse)).all(), (what, off.max())
            scales = cache4.bf16_value(v4[b, u, at].cpu().numpy()[:, 64:].reshape(-1, 4, 4)[..., :2]
                                       .copy().view(np.uint16)[..., 0].astype(np.uint32))
            scales = np.repeat(scales, 32, axis=1)
            with np.errstate(divide="ignore", invalid="ignore"):
                code = np.where(scales > 0, -vlo / scales, 0.0)
            near = np.abs(code - np.floor(code) - 0.5) < 2.0 ** -16
            mid = vlo + scales * np.clip(np.rint(code), 0, 15)
            A = p @ (np.abs(V - mid) + near * scales)
            bound = 2.0 ** -8 * ((1 + 2.0 ** -6) * A + np.abs(ref)) + (
                2 * E[:, None] + 2.0 ** -20) * (p @ (np.abs(vlo) + np.abs(V)) + np.abs(ref))
            err = np.abs(o[b, 0, u * g:u * g + g] - ref)
            assert (err <= bound).all(), (what, (err - bound).max())


STEP = [
    # B, C, n_q, n_kv, lens, window, sinks
    (1, 1, 1, 1, [1], None, 0),
    (1, 1, 4, 1, [0], None, 0),
    (1, 40, 4, 1, [16], None, 0),
    (3, 333, 10, 5, [333, 100, 0], None, 0),
    (5, 300, 4, 4, [15, 16, 17, 31, 33], None, 0),
    (4, 2000, 8, 1, [2000, 1, 1999, 640], None, 0),              # g = 8
    (2, 1500, 9, 1, [1500, 77], None, 0),                        # g = 9: two tiles of heads
    (2, 2000, 12, 1, [77, 1999], None, 0),
    (2, 1000, 32, 2, [1000, 511], None, 0),                      # g = 16
    (1, 20000, 36, 6, [19999], None, 0),
    (1, 30000, 2, 1, [30000], None, 0),                          # every CTA on one head
    (6, 700, 16, 8, [0, 0, 0, 5, 0, 0], None, 0),
    (3, 50, 8, 2, [0, 0, 0], None, 0),
    (40, 260, 14, 2, [(37 * i) % 261 for i in range(40)], None, 0),
    (300, 140, 4, 2, [(53 * i) % 141 for i in range(300)], None, 0),
    (3, 333, 10, 5, [333, 100, 0], 64, 4),
    (5, 600, 4, 4, [15, 16, 17, 385, 600], 16, 0),
    (4, 900, 8, 1, [900, 1, 899, 640], 1, 1),
    (2, 900, 12, 1, [900, 77], 400, 300),
    (3, 300, 8, 2, [300, 299, 1], 10 ** 12, 10 ** 12),
    (2, 40000, 16, 2, [39999, 5], 4096, 130),
]


def make_step(B, C, n_q, n_kv, lens, window, sinks, seed=0):
    """Caches with NaN scales and lowest values wherever no token looks."""
    q = W.make_inputs(W.custom(B, 1, n_q, n_kv, 128, Lk=4), "cuda", seed=seed)[0]
    caches = []
    for i in range(2):
        c = torch.full((B, n_kv, C, 80), 255, dtype=torch.uint8, device="cuda")
        x = rows(B, C, n_kv, seed + i, "outliers" if i == 0 else "normal")
        for b in range(B):
            n = min(max(lens[b], 0), C)
            first = max(0, n - window) if window else 0
            at = [*range(min(sinks, first)), *range(first, n)]
            packed = torch.from_numpy(cache4.pack(x[b, at].double().cpu().numpy())).cuda()
            c[b, :, at] = packed.transpose(0, 1)
        caches.append(c)
    return q, *caches, i32(*lens)


@pytest.mark.parametrize("case", STEP, ids=lambda c: "B%d_C%d_q%d_kv%d_W%s_S%d" % (c[:4] + c[5:]))
def test_decode(case):
    q, k4, v4, lens = make_step(*case, seed=case[0] + case[1])
    o, lse = attn_decode4(q, k4, v4, lens, window=case[5], sinks=case[6])
    assert attn_device_check() == ATTN_OK
    check_step(q, k4, v4, case[4], o, lse, *case[5:], what=str(case[:4]))


def test_decode_random_shapes():
    rng = np.random.default_rng(23)
    for n in range(40):
        n_kv = int(rng.choice([1, 2, 3, 5]))
        n_q = n_kv * int(rng.choice([1, 2, 4, 7, 8, 11, 16]))
        B, C = int(rng.integers(1, 9)), int(rng.integers(1, 700))
        window = int(rng.integers(1, 400)) if n % 3 else None
        sinks = int(rng.choice([0, 1, 4, rng.integers(0, 300)])) if window else 0
        lens = [int(x) for x in rng.integers(-2, C + 3, B)]
        q, k4, v4, t = make_step(B, C, n_q, n_kv, lens, window, sinks, seed=n)
        o, lse = attn_decode4(q, k4, v4, t, window=window, sinks=sinks)
        check_step(q, k4, v4, lens, o, lse, window, sinks, what=str((B, C, n_q, n_kv, window, sinks)))
    assert attn_device_check() == ATTN_OK


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_decode_other_scales(scale):
    q, k4, v4, lens = make_step(2, 500, 8, 2, [500, 123], None, 0, seed=9)
    o, lse = attn_decode4(q, k4, v4, lens, scale=scale)
    check_step(q, k4, v4, [500, 123], o, lse, None, 0, scale=scale)


@pytest.mark.parametrize("kind", ["normal", "outliers"])
def test_decode_of_long_caches_is_as_exact_as_its_roundings(kind):
    """Over long caches of values around 0, O is small beside them, and what the weights'
    roundings do must shrink with it: two roundings of up to half a bf16 step, 2^-8 /
    sqrt(3) in the mean at most, one on O and one on V less the code's value next to 0,
    which in the mean square is larger than V by what half a step is at most, a tenth
    for groups of normal values and less for outliers: sqrt(2 / 3) 1.1 2^-8 of O."""
    B, C, n_q, n_kv = 2, 6000, 8, 2
    lens = [6000, 3500]
    k, v = rows(B, C, n_kv, 30), rows(B, C, n_kv, 31, kind)
    k4, v4 = (torch.zeros(B, n_kv, C, 80, dtype=torch.uint8, device="cuda") for _ in range(2))
    attn_pack4(k, v, k4, v4)
    q = W.make_inputs(W.custom(B, 1, n_q, n_kv, 128, Lk=4), "cuda", seed=32)[0]
    o = to_np(attn_decode4(q, k4, v4, i32(*lens))[0])
    err = size = 0.0
    for b in range(B):
        for h in range(n_q):
            K, V = (cache4.unpack(c[b, h // 4, :lens[b]].cpu().numpy())[0] for c in (k4, v4))
            s = K @ to_np(q)[b, 0, h] * 128 ** -0.5
            p = np.exp(s - s.max())
            ref = p @ V / p.sum()
            err, size = err + ((o[b, 0, h] - ref) ** 2).sum(), size + (ref ** 2).sum()
    assert (err / size) ** 0.5 <= (2 / 3) ** 0.5 * 1.1 * 2.0 ** -8


def test_decode_what_is_not_a_number_stays_in_its_head():
    q, k4, v4, lens = make_step(2, 3000, 8, 2, [3000, 2000], None, 0, seed=10)
    o, lse = attn_decode4(q, k4, v4, lens)
    bad = k4.clone()
    bad[1, 0, 700, 64:] = 255
    o2, lse2 = attn_decode4(q, bad, v4, lens)
    assert o2[1, 0, :4].isnan().all() and lse2[1, :4].isnan().all()
    assert torch.equal(o2[0], o[0]) and torch.equal(o2[1, 0, 4:], o[1, 0, 4:])
    bad = v4.clone()
    bad[1, 1, 700, 68:72] = 255                      # one group of one row of V
    o3, lse3 = attn_decode4(q, k4, bad, lens)
    assert o3[1, 0, 4:, 32:64].isnan().all() and torch.equal(lse3, lse)
    o3[1, 0, 4:, 32:64] = o[1, 0, 4:, 32:64]
    assert torch.equal(o3, o)


def test_decode_same_bits_again_and_one_workspace():
    ws = torch.full((attn_decode4_workspace_bytes(4, 3000, 8, 2),), 255, dtype=torch.uint8,
                    device="cuda")
    q, k4, v4, lens = make_step(4, 3000, 8, 2, [3000, 17, 0, 2222], None, 0, seed=11)
    first = attn_decode4(q, k4, v4, lens, workspace=ws)
    for _ in range(3):
        again = attn_decode4(q, k4, v4, lens, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    with pytest.raises(AttnError):
        attn_decode4(q, k4, v4, lens, workspace=ws[:-1])


def test_a_prompt_and_its_steps():
    """A prompt's rows stored, steps that append their own row, the whole read back."""
    B, n_q, n_kv, C = 2, 8, 2, 90
    k, v = rows(B, 80, n_kv, 12), rows(B, 80, n_kv, 13)
    k4, v4 = (torch.zeros(B, n_kv, C, 80, dtype=torch.uint8, device="cuda") for _ in range(2))
    lens = i32(70, 33)
    attn_pack4(k[:, :70].contiguous(), v[:, :70].contiguous(), k4, v4, counts=lens)
    for i in range(70, 80):
        attn_pack4(k[:, i:i + 1].contiguous(), v[:, i:i + 1].contiguous(), k4, v4, lens)
        lens += 1
        q = W.make_inputs(W.custom(B, 1, n_q, n_kv, 128, Lk=4), "cuda", seed=i)[0]
        o, lse = attn_decode4(q, k4, v4, lens, window=50, sinks=2)
        check_step(q, k4, v4, lens.tolist(), o, lse, 50, 2, what=str(i))
    want = stored(torch.zeros(B, n_kv, C, 80, dtype=torch.uint8), k, [0, 0], [80, 33])
    want[1, :, 33:43] = cache4.pack(k[1, 70:80].double().cpu().numpy()).transpose(1, 0, 2)
    assert np.array_equal(k4.cpu().numpy(), want)
