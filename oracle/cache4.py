"""fp64 reference of caches held in 4 bits: rows into codes and back.

TEST INFRASTRUCTURE ONLY, like the rest of this package: written from the
format, group by group.

    group g of a row: channels 32 g .. 32 g + 31; lo = min, scale = (max - lo) / 15
    rounded to fp32 and then bf16; code = rint((x - lo) / scale), at most 15
    byte 4 (4 t + g) + i / 2 holds the codes of channels 32 g + 8 t + i, even i low
    bytes 64 + 4 g ..: scale, lo (bf16, little endian)
"""

from __future__ import annotations

import numpy as np


def bf16_bits(x):
    """The bf16 nearest to fp32 values (ties to even), as uint16; NaN as 0x7FC0."""
    x = np.asarray(x, dtype=np.float32)
    b = x.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_value(bits):
    with np.errstate(invalid="ignore"):                   # (signalling NaNs)
        return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)


def pack(x):
    """Rows x [..., 128] (values of bf16, as float64) -> uint8 [..., 80]."""
    out = np.zeros(x.shape[:-1] + (80,), dtype=np.uint8)
    for g in range(4):
        v = x[..., 32 * g:32 * g + 32]
        finite = np.isfinite(v).all(-1)
        v = np.where(finite[..., None], v, 0.0)
        lo = v.min(-1)
        sb = bf16_bits(((v.max(-1) - lo) / 15).astype(np.float32))
        s = bf16_value(sb)
        q = (v - lo[..., None]) / np.where(s > 0, s, 1.0)[..., None]
        code = np.where((s > 0)[..., None], np.minimum(np.rint(q), 15), 0).astype(np.uint8)
        code = np.where(finite[..., None], code, 0)
        for t in range(4):
            for i in range(8):
                out[..., 4 * (4 * t + g) + i // 2] |= code[..., 8 * t + i] << (4 * (i % 2))
        lob = np.where(finite, bf16_bits(lo.astype(np.float32)), np.uint16(0x7FC0))
        sb = np.where(finite, sb, np.uint16(0x7FC0))
        for at, word in ((64 + 4 * g, sb), (66 + 4 * g, lob)):
            out[..., at] = word & 255
            out[..., at + 1] = word >> 8
    return out


def parts(rows):
    """(lo, scale * code) [..., 128] of rows of 80 bytes, both exact."""
    low, product = np.zeros(rows.shape[:-1] + (128,)), np.zeros(rows.shape[:-1] + (128,))
    word = lambda at: rows[..., at].astype(np.uint32) | (rows[..., at + 1].astype(np.uint32) << 8)  # noqa: E731
    for g in range(4):
        s, lo = bf16_value(word(64 + 4 * g)), bf16_value(word(66 + 4 * g))
        for t in range(4):
            for i in range(8):
                code = (rows[..., 4 * (4 * t + g) + i // 2] >> (4 * (i % 2))) & 15
                with np.errstate(invalid="ignore"):       # (an infinite scale times 0)
                    product[..., 32 * g + 8 * t + i] = s * code
                low[..., 32 * g + 8 * t + i] = lo
    return low, product


def unpack(rows):
    """(values [..., 128], lo of each value's group [..., 128]) that rows stand for."""
    low, product = parts(rows)
    with np.errstate(invalid="ignore"):
        return low + product, low


def rounded(rows):
    """The values rounded once to bf16 (ties to even, infinite beyond its range).

    lo and scale * code may be so far apart that their fp64 sum drops bits; those
    only matter where the sum is half-way between two bf16."""
    low, product = parts(rows)
    with np.errstate(invalid="ignore"):
        x = low + product
        back = x - low
        left = (low - (x - back)) + (product - back)      # x + left is the exact sum
    sane = np.isfinite(x)
    y = np.where(sane, x, 0.0)
    ulp = np.ldexp(1.0, np.maximum(np.frexp(y)[1], -125) - 8)   # 8 bits; 2^-133 at least
    q = y / ulp
    down = np.floor(q)
    up = np.where(q - down == 0.5, np.where(left == 0, down % 2 == 1, left > 0), q - down > 0.5)
    y = (down + up) * ulp
    return np.where(sane, np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, y), y), x)
