"""Caches held in 4 bits, on the CPU: the format's fp64 reference in closed form
and against bounds, and what the calls refuse before any CUDA call."""

import math

import numpy as np
import pytest

import causal_gqa_prefill_gb300 as cg
from oracle import cache4

INVALID, UNSUPPORTED = cg.ATTN_ERR_INVALID_ARG, cg.ATTN_ERR_UNSUPPORTED


def _bf16(x):
    return cache4.bf16_value(cache4.bf16_bits(x))


def test_bf16_against_torch():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(0).standard_normal(4000).astype(np.float32)
    x = np.concatenate([x, x * np.float32(1e-39), x * np.float32(1e37), [0.0, -0.0, np.inf, -np.inf]])
    x = x.astype(np.float32)
    t = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(cache4.bf16_bits(x), t)


def test_a_row_counted_out():
    """Channels 0 .. 15 twice in every group: lo 0, scale 1, the codes themselves."""
    row = np.tile(np.arange(16.0), 8)
    b = cache4.pack(row)
    assert b.shape == (80,)
    for g in range(4):
        for t in range(4):
            word = int.from_bytes(b[4 * (4 * t + g):4 * (4 * t + g) + 4].tobytes(), "little")
            assert [(word >> 4 * i) & 15 for i in range(8)] == [(8 * t + i) % 16 for i in range(8)]
        assert b[64 + 4 * g:68 + 4 * g].tolist() == [0x80, 0x3F, 0, 0]
    assert np.array_equal(cache4.unpack(b)[0], row)


def test_values_are_within_half_a_step():
    x = _bf16(np.random.default_rng(1).standard_normal((50, 128)) * 3)
    val, low = cache4.unpack(cache4.pack(x))
    g = x.reshape(50, 4, 32)
    scale = _bf16((g.max(-1) - g.min(-1)) / 15)
    # half a step, and at the top what the scale's rounding (2^-8 of it) cuts off of 15 steps
    assert (np.abs(val - x).reshape(50, 4, 32) <= (0.5 + 15 * 2.0 ** -8) * scale[..., None]).all()
    assert np.array_equal(low.reshape(50, 4, 32)[..., 0], g.min(-1))


def test_constant_groups_and_what_is_not_finite():
    x = np.zeros((3, 128))
    x[0, :32], x[1, 40], x[2, 100], x[2, 64:96] = -2.5, np.nan, np.inf, np.arange(32) % 16
    val, _ = cache4.unpack(cache4.pack(x))
    assert np.array_equal(val[0], x[0])
    assert np.isnan(val[1, 32:64]).all() and not val[1, 64:].any() and not val[1, :32].any()
    assert np.isnan(val[2, 96:]).all() and np.array_equal(val[2, 64:96], x[2, 64:96])


def test_rounded_once():
    """Random bytes: exact fractions decide which bf16 a value goes to."""
    from fractions import Fraction

    rows = np.random.default_rng(5).integers(0, 256, (40, 80)).astype(np.uint8)
    low, product = cache4.parts(rows)
    got = cache4.rounded(rows)
    checked = 0
    for lo, p, y in zip(low.ravel(), product.ravel(), got.ravel()):
        if not np.isfinite(lo + p) or not np.isfinite(y):
            continue
        exact = Fraction(lo) + Fraction(p)
        bits = int(cache4.bf16_bits(np.float32(y)))
        assert float(cache4.bf16_value(np.uint16(bits))) == y
        for n in (bits - 1, bits + 1):                 # the neighbours are no nearer
            if bits & 0x7FFF and (n & 0x7FFF) < 0x7F80:
                other = abs(Fraction(float(cache4.bf16_value(np.uint16(n)))) - exact)
                own = abs(Fraction(y) - exact)
                assert own < other or (own == other and bits % 2 == 0)
        checked += 1
    assert checked > 4000


def test_ties_go_to_the_even_code():
    row = np.tile(np.concatenate([[0.0, 15.0, 0.5, 1.5, 2.5, 13.5, 14.5], np.ones(25)]), 4)
    val, _ = cache4.unpack(cache4.pack(row))
    assert val[:7].tolist() == [0, 15, 0, 2, 2, 14, 14]


# ------------------------------------------------------------------ refusals

FAKE = 1 << 20   # 16-byte aligned, never dereferenced: each call fails validation first
FAR = [FAKE + i * (1 << 40) for i in range(4)]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from causal_gqa_prefill_gb300 import build
    build.build()


ROWS = [(dict(k=0), INVALID), (dict(v4=0), INVALID), (dict(k=FAR[0] + 8), INVALID),
        (dict(k4=FAR[2] + 4), INVALID), (dict(at=FAKE + 2), INVALID), (dict(B=0), INVALID),
        (dict(L=0), INVALID), (dict(C=0), INVALID), (dict(n_kv=0), INVALID),
        (dict(d_h=64), UNSUPPORTED), (dict(L=1 << 31), UNSUPPORTED), (dict(C=1 << 31), UNSUPPORTED),
        (dict(B=1 << 25), UNSUPPORTED), (dict(k4=FAR[3]), INVALID)]


@pytest.mark.parametrize("args,expect", ROWS)
def test_row_refusals(args, expect):
    a = dict(k=FAR[0], v=FAR[1], k4=FAR[2], v4=FAR[3], at=FAKE, B=2, L=3, C=10, n_kv=2, d_h=128)
    a.update(args)
    assert cg.attn_cache_pack4(**a, counts=0, stream=0) == expect
    if "k4" not in args or args["k4"] != FAR[3]:    # (reading one cache twice is allowed)
        assert cg.attn_cache_unpack4(**a, stream=0) == expect


def test_overlaps_are_refused():
    rows, held = 2 * 3 * 2 * 256, 2 * 2 * 10 * 80
    sizes = (2, 3, 10, 2, 128, 0)
    assert cg.attn_cache_pack4(FAR[0], FAR[1], FAR[0] + rows - 16, FAR[3], 0, 0, *sizes) == INVALID
    assert cg.attn_cache_pack4(FAR[0], FAR[1], FAR[2], FAR[2] + held - 16, 0, 0, *sizes) == INVALID
    assert cg.attn_cache_unpack4(FAR[2], FAR[3], FAR[2] + held - 16, FAR[1], 0, *sizes) == INVALID
    assert cg.attn_cache_unpack4(FAR[2], FAR[3], FAR[0], FAR[0], 0, *sizes) == INVALID


STEP = [(dict(q=0), INVALID), (dict(k4=FAKE + 8), INVALID), (dict(lens=FAKE + 1), INVALID),
        (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(window=0, sinks=3), INVALID),
        (dict(C=0), INVALID), (dict(n_q=5), INVALID), (dict(n_q=34), UNSUPPORTED),
        (dict(d_h=64), UNSUPPORTED), (dict(C=1 << 31), UNSUPPORTED),
        (dict(workspace_bytes=100), INVALID), (dict(scale=math.inf), INVALID)]


@pytest.mark.parametrize("args,expect", STEP)
def test_step_refusals(args, expect):
    a = dict(q=FAKE, k4=FAKE, v4=FAKE, lens=FAKE, o=FAKE, lse=FAKE, workspace=FAKE,
             workspace_bytes=1 << 40, B=1, C=128, n_q=4, n_kv=2, d_h=128, window=16, sinks=2,
             scale=0.125)
    a.update(args)
    assert cg.attn_decode4_fwd(**a, stream=0) == expect


def test_step_workspace():
    size = cg.attn_decode4_workspace_bytes
    assert size(1, 1 << 17, 8, 2) > size(1, 1 << 17, 8, 2, window=64) > 0
    # two places per head and CTA, whatever the length
    assert size(1, 1 << 30, 8, 2) <= 2 * (2 + 152) * 4 * (512 + 8) + 1024
    for bad in (dict(window=0, sinks=1), dict(d_h=64), dict(window=-1)):
        assert size(1, 100, 8, 2, **bad) == -1


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    c = torch.zeros(1, 2, 9, 80, dtype=torch.uint8)
    for call in (lambda: cg.attn_pack4(x, x, c, c), lambda: cg.attn_unpack4(c, c, 3),
                 lambda: cg.attn_decode4(x[:, :1], c, c, x)):
        with pytest.raises(TypeError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="length"):
        cg.attn_unpack4(c, c, 0)
    with pytest.raises(ValueError, match="window"):
        cg.attn_decode4(x[:, :1], c, c, x, sinks=2)
    with pytest.raises(ValueError, match="window"):
        cg.attn_decode4(x[:, :1], c, c, x, window=0)
