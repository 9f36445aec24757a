"""Plain float64 definition of the 4-bit paged key / value cache and of
single-token attention over it.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path imports this module.

A row is cut into groups of 32 elements.  A group's scale is the smallest
number m * 2^e with m in 8..15 and e in -17..12 (or m in 0..7 at e = -17) that
is not below max|x| / 7, at most 61440; its byte is 8 * (e + 17) + m for e =
-17, else 8 * (e + 18) + (m - 8): the bits 7..14 of the same number in fp16.  A
group with NaN or an infinity has the byte 255 and reads as NaN.  Codes are
8 + rint(x / scale), clamped to 1..15; code n stands for (n - 8) * scale.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

from .hysparse import attend, first_window_key_set

__all__ = ["scale_of", "byte_value", "quantise", "values", "page_bytes", "pack_row",
           "unpack_row", "positions", "decode"]

_SCALES = [Fraction(m, 1) * Fraction(2) ** -17 for m in range(8)] + [
    Fraction(m) * Fraction(2) ** e for e in range(-17, 13) for m in range(8, 16)]


def scale_of(amax: float):
    """(byte, scale) of a group whose largest magnitude is ``amax``, in exact
    arithmetic over the ordered list of every scale."""
    a = Fraction(float(amax))
    lo, hi = 0, len(_SCALES) - 1
    while lo < hi:  # the first scale with 7 * scale >= amax, else the last
        mid = (lo + hi) // 2
        if 7 * _SCALES[mid] >= a:
            hi = mid
        else:
            lo = mid + 1
    return lo, float(_SCALES[lo])


def byte_value(byte: int) -> float:
    return float("nan") if byte >= len(_SCALES) else float(_SCALES[byte])


def quantise(x):
    """x [n, D] -> (codes uint8 [n, D], scale bytes uint8 [n, D / 32])."""
    x = np.asarray(x, np.float64)
    n, D = x.shape
    codes = np.full((n, D), 8, np.uint8)
    byte = np.zeros((n, D // 32), np.uint8)
    for i in range(n):
        for g in range(D // 32):
            v = x[i, 32 * g:32 * g + 32]
            if not np.all(np.isfinite(v)):
                byte[i, g] = 255
                continue
            byte[i, g], s = scale_of(np.abs(v).max())
            if s > 0:
                codes[i, 32 * g:32 * g + 32] = (8 + np.clip(np.rint(v / s), -7, 7)).astype(np.uint8)
    return codes, byte


def values(codes, byte):
    s = np.asarray([[byte_value(int(b)) for b in row] for row in byte], np.float64)
    return (codes.astype(np.float64) - 8) * np.repeat(s.reshape(len(codes), -1), 32, axis=1)


# ------------------------------------------------------------------ pages
def page_bytes(width: int, page_size: int) -> int:
    g = width // 32
    return page_size * (16 * g + 4 * ((g + 3) // 4))


def _offsets(width, page_size, slot):
    G = width // 32
    code = [(g * page_size + slot) * 16 for g in range(G)]
    scale = [G * page_size * 16 + ((g // 4) * page_size + slot) * 4 + g % 4 for g in range(G)]
    return code, scale


def pack_row(page, width, page_size, slot, codes, byte):
    """Writes one row into ``page`` (uint8 [page_bytes])."""
    code_at, scale_at = _offsets(width, page_size, slot)
    for g in range(width // 32):
        for w in range(4):
            word = 0
            for e in range(8):
                word |= int(codes[32 * g + 8 * w + e]) << (4 * (e // 2) + 16 * (e % 2))
            for b in range(4):
                page[code_at[g] + 4 * w + b] = (word >> (8 * b)) & 255
        page[scale_at[g]] = byte[g]


def unpack_row(page, width, page_size, slot):
    """float64 values of one row of ``page``."""
    code_at, scale_at = _offsets(width, page_size, slot)
    codes = np.empty((1, width), np.uint8)
    byte = np.empty((1, width // 32), np.uint8)
    for g in range(width // 32):
        byte[0, g] = page[scale_at[g]]
        for w in range(4):
            word = sum(int(page[code_at[g] + 4 * w + b]) << (8 * b) for b in range(4))
            for e in range(8):
                codes[0, 32 * g + 8 * w + e] = (word >> (4 * (e // 2) + 16 * (e % 2))) & 15
    return values(codes, byte)[0]


# ------------------------------------------------------------------ decode
def positions(length: int, window: int, first: int):
    """Cached positions a query at length - 1 attends (window 0: all)."""
    if length == 0:
        return np.zeros(0, np.int64)
    return (np.arange(length) if window == 0
            else first_window_key_set(length - 1, 0, window, first))


def decode(q, k_rows, v_rows, window: int, first: int, sink=None, scale=None):
    """q [S, H, Dk]; k_rows[s] [len, Dk], v_rows[s] [len, Dv]: the cached values
    of sequence s.  Returns (out [S, H, Dv], lse [S, H])."""
    q = np.asarray(q, np.float64)
    sc = q.shape[2] ** -0.5 if scale is None else scale
    got = [attend(q[s], positions(len(k), window, first), k, v, sink, sc)
           for s, (k, v) in enumerate(zip(k_rows, v_rows))]
    return np.stack([g[0] for g in got]), np.stack([g[1] for g in got])
