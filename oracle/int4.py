"""Oracle: 4-bit cached values and their layout (test infrastructure only).

A token's row of one head is stored in groups of 16 elements.  A group with largest magnitude
``amax`` has the scale ``min(amax / 7, 896)`` rounded to nearest even on the grid of an unsigned
float with 5 exponent bits (bias 15) and 3 mantissa bits; each element is the code ``x / scale``
rounded to nearest even and clamped to -7 .. 7 (scale 0: code 0), and stands for ``code * scale``.
A group with a NaN has the scale byte 0xFF (NaN).

Quotients are taken in float32 from float32 inputs (``numpy`` divides correctly rounded), which
is what the definition in the library's header rounds; ``quantize64`` takes them in float64.

Layout of one (block, head) tile, per 8 tokens: ``4 * d`` bytes of codes, then ``d / 2`` scale
bytes.  K codes ``[token][d/2]`` bytes, element 2i in byte i's low nibble; K scales
``[token][d/16]``.  V codes in 16-bit pieces of 4 elements of one token (element i of the piece at
bits 4i), ``[chunk of d/8 elements][token/2][d/32][token%2]``; V scales ``[d/16][token]``.
"""

from __future__ import annotations

import math

import numpy as np

MAX_SCALE = 896.0
NAN_BYTE = 0xFF


def decode_scale(byte: int) -> float:
    """Value of one scale byte (exact)."""
    e, m = int(byte) >> 3, int(byte) & 7
    if e == 31:
        return math.nan if m else math.inf
    return math.ldexp(m, -17) if e == 0 else math.ldexp(8 + m, e - 18)


SCALES = np.array([decode_scale(b) for b in range(256)])


def encode_scale(s: float) -> int:
    """The byte nearest to s >= 0 (halves to the even byte), s at most 896."""
    s = min(float(s), MAX_SCALE)
    table = SCALES[:248]                               # finite values, increasing
    i = int(np.searchsorted(table, s))
    if table[i] == s:
        return i
    lo, hi = table[i - 1], table[i]
    if s - lo != hi - s:
        return i - 1 if s - lo < hi - s else i
    return i - 1 if (i - 1) % 2 == 0 else i


def quantize(rows, quotient=np.float32):
    """rows [..., d] -> (codes int8 [..., d] in -7 .. 7, scale bytes uint8 [..., d/16])."""
    x = np.asarray(rows).astype(quotient)
    g = x.reshape(*x.shape[:-1], -1, 16)
    top = np.max(np.abs(g), axis=-1)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        s = (top / quotient(7.0)).astype(quotient)
        byte = np.array([NAN_BYTE if math.isnan(v) else encode_scale(v) for v in s.reshape(-1)],
                        dtype=np.uint8).reshape(s.shape)
        v = SCALES[byte].astype(quotient)[..., None]
        q = np.where(v > 0, g / np.where(v > 0, v, quotient(1)), quotient(0))
        q = np.clip(np.rint(q), -7, 7)
    return np.where(np.isnan(q), 0, q).astype(np.int8).reshape(x.shape), byte


def quantize64(rows):
    return quantize(rows, np.float64)


def dequantize(codes, scale_bytes) -> np.ndarray:
    """float64 values of codes [..., d] with scale bytes [..., d/16]."""
    c = np.asarray(codes, dtype=np.float64)
    s = SCALES[np.asarray(scale_bytes)]
    return (c.reshape(*c.shape[:-1], -1, 16) * s[..., None]).reshape(c.shape)


def store(pool, which: str, block: int, head: int, offset: int, codes, scale_bytes) -> None:
    """Put one token's codes and scale bytes into a pool [blocks, H, B/8, 4d + d/2] (uint8)."""
    d = len(codes)
    oct_ = pool[block, head, offset // 8]
    t = offset % 8
    for e in range(d):
        nib = int(codes[e]) + 8
        if which == "k":
            byte, high = t * (d // 2) + e // 2, e % 2
        else:
            chunk, i = divmod(e, d // 8)
            piece = ((chunk * 4 + t // 2) * (d // 32) + i // 4) * 2 + t % 2
            byte, high = 2 * piece + (i % 4) // 2, e % 2
        old = int(oct_[byte])
        oct_[byte] = (old & 0x0F) | (nib << 4) if high else (old & 0xF0) | nib
    for g in range(d // 16):
        oct_[4 * d + (t * (d // 16) + g if which == "k" else g * 8 + t)] = scale_bytes[g]


def load(pool, which: str, block: int, head: int, offset: int, d: int):
    """The token's (codes, scale bytes) back from a pool."""
    oct_ = pool[block, head, offset // 8]
    t = offset % 8
    codes = np.empty(d, dtype=np.int8)
    for e in range(d):
        if which == "k":
            byte = t * (d // 2) + e // 2
        else:
            chunk, i = divmod(e, d // 8)
            byte = 2 * (((chunk * 4 + t // 2) * (d // 32) + i // 4) * 2 + t % 2) + (i % 4) // 2
        v = int(oct_[byte])
        codes[e] = (v >> 4 if e % 2 else v & 15) - 8
    scales = np.array([oct_[4 * d + (t * (d // 16) + g if which == "k" else g * 8 + t)] for g in range(d // 16)],
                      dtype=np.uint8)
    return codes, scales


def token_values(pool, which: str, d: int, blocks, offsets) -> np.ndarray:
    """float64 [n, H, d] of many tokens (vectorised; agrees with ``load`` element by element)."""
    blocks, offsets = np.asarray(blocks), np.asarray(offsets)
    e = np.arange(d)[None]
    t = (offsets % 8)[:, None]
    if which == "k":
        byte, scale = t * (d // 2) + e // 2, t * (d // 16) + e // 16
    else:
        chunk, i = e // (d // 8), e % (d // 8)
        byte = 2 * (((chunk * 4 + t // 2) * (d // 32) + i // 4) * 2 + t % 2) + (i % 4) // 2
        scale = (e // 16) * 8 + t
    octs = pool[blocks, :, offsets // 8]                              # [n, H, 4d + d/2]
    b = np.take_along_axis(octs, np.broadcast_to(byte[:, None], octs.shape[:2] + (d,)), 2)
    s = np.take_along_axis(octs, np.broadcast_to(4 * d + scale[:, None], octs.shape[:2] + (d,)), 2)
    nib = np.where(e % 2 == 1, b >> 4, b & 15).astype(np.float64)
    return (nib - 8.0) * SCALES[s]
