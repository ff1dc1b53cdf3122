"""Rows of a paged cache in 4 bits: E2M1 codes with a bfloat16 scale for every
16 values, as records of bytes; in float64 where a number is a value.

Test infrastructure only (see the package docstring).  The format is the
library's own (include/dflash.h, "Paged cache"; the pages serve their models in
NVFP4 among others, product doc "Speculative decoding", introduction, without
saying how a cache is held).
"""

import numpy as np

BLOCK = 16
# sign apart, the eight values: subnormals 0 and 1/2 of exponent field 0, then
# (1 + m / 2) 2^(e - 1)
MAGNITUDE = np.array([m / 2.0 if e == 0 else (1.0 + m / 2.0) * 2.0 ** (e - 1) for e in range(4) for m in range(2)])


def value(code):
    """Real value of 4-bit codes."""
    c = np.asarray(code).astype(np.int64)
    return MAGNITUDE[c & 7] * np.where(c & 8, -1.0, 1.0)


def round_code(x):
    """Codes of values x: the nearest magnitude, ties to the even index, 6 at
    most; the sign kept.  NaN has no code (0 here)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 6.0)
    d = np.abs(a[..., None] - MAGNITUDE)
    near = d == d.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1) & (near.sum(axis=-1) > 1), even.argmax(axis=-1), near.argmax(axis=-1))
    return np.where(np.isnan(x), 0, code | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def bf16_bits(x):
    """float32 values rounded to nearest bfloat16, ties to even, as uint16."""
    b = np.ascontiguousarray(np.asarray(x, dtype=np.float32)).view(np.uint32).astype(np.uint64)
    r = (b + 0x7FFF + ((b >> 16) & 1)) >> 16
    return np.where(np.isnan(x), 0x7FC0, r).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def scales(x):
    """Scales (float64, bfloat16 values) of rows x [..., hd] (float32 values):
    max / 6 as a float32 quotient, rounded; 1 where that is 0, NaN where the
    block is not finite."""
    b = np.asarray(x, dtype=np.float32).reshape(x.shape[:-1] + (-1, BLOCK))
    bad = ~np.isfinite(b).all(axis=-1)
    s = bf16_value(bf16_bits(np.where(bad, 0, np.abs(np.where(np.isfinite(b), b, 0)).max(axis=-1)) / np.float32(6)))
    return np.where(bad, np.nan, np.where(s == 0, 1.0, s))


def pack(x):
    """Records (uint8 [..., hd * 5 / 8]) of rows x [..., hd]."""
    x = np.asarray(x, dtype=np.float32)
    s = scales(x)
    with np.errstate(invalid="ignore", over="ignore"):
        y = x.reshape(s.shape + (BLOCK,)) / s.astype(np.float32)[..., None]
    c = round_code(np.where(y == 0, 0.0, y)).reshape(x.shape)       # -0 becomes 0
    bits = bf16_bits(s.astype(np.float32))
    two = np.stack([bits & 0xFF, bits >> 8], -1).astype(np.uint8).reshape(x.shape[:-1] + (-1,))
    return np.concatenate([c[..., 0::2] | (c[..., 1::2] << 4), two], -1)


def split(records):
    """(codes [..., hd], scales [..., hd / 16] float64) of records."""
    r = np.asarray(records)
    hd = r.shape[-1] * 8 // 5
    low = r[..., :hd // 2]
    codes = np.stack([low & 15, low >> 4], -1).reshape(r.shape[:-1] + (hd,))
    b = r[..., hd // 2:].astype(np.uint16)
    return codes, bf16_value(b[..., 0::2] | (b[..., 1::2] << 8))


def unpack(records):
    """Rows of records, float64 [..., hd]."""
    codes, s = split(records)
    return value(codes) * np.repeat(s, BLOCK, axis=-1)


def sequence(pages, table_row, length, page):
    """Positions 0 .. length - 1 of one request, [length, heads, hd] float64:
    pages [n_pages, heads, page, hd * 5 / 8] as uint8."""
    at = np.arange(length)
    return unpack(np.asarray(pages)[np.asarray(table_row)[at // page], :, at % page])
