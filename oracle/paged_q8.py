"""Paged caches in 8 bits and norms of heads (oracle, float64).

What it restates
  * The blog's cache handling over a cache of e4m3 codes (OCP 8-bit floating point: 4 exponent
    bits of bias 7, 3 mantissa bits, largest 448, code 127 no number) whose rows share a
    power-of-two scale in blocks: number = code * 2^(s - 127), s a byte for each page, KV head and
    block of `blk` rows.
  * The norm of a head: x -> w x / sqrt(mean of x^2 + eps).

Readings (not fixed by the pages)
  * A block that receives rows takes the least scale, 2^-117 or more, under which none of them
    exceeds 448; what is not finite does not count and becomes no number.  A block that begins with
    committed rows keeps at least its scale, and those rows are coded anew where it grows.
  * A commit gives a block that receives rows the largest of its scale and those that the rows
    had; its rows up to the path's end are coded for it, the others' bytes stay.
"""
from __future__ import annotations

import numpy as np

LEAST = -117
_POS = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7) for e in range(16)
                 for m in range(8)][:127])  # codes 0..126; 127 is no number


def decode(codes):
    c = np.asarray(codes, dtype=np.uint8)
    table = np.concatenate((_POS, [np.nan], -_POS, [np.nan]))
    return table[c]


def encode(x):
    """Codes of the nearest e4m3 numbers, ties to the even code; not finite: 127."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.abs(x)
    mid = (_POS[1:] + _POS[:-1]) / 2
    lo = np.searchsorted(mid, mag, side="left")  # a tie: the lower code
    tie = (lo < mid.size) & (mag == mid[np.minimum(lo, mid.size - 1)])
    lo = lo + (tie & (lo % 2 == 1))
    out = np.where(np.signbit(x), lo + 128, lo)
    return np.where(np.isfinite(x), out, 127).astype(np.uint8)


def exponent(rows):
    """Least e >= LEAST under which no finite entry exceeds 448."""
    mag = np.abs(np.asarray(rows, dtype=np.float64))
    top = float(np.max(mag[np.isfinite(mag)], initial=0.0))
    e = LEAST
    while top > 448.0 * 2.0 ** e:
        e += 1
    return e


def numbers(codes, scale):
    """The numbers of a cache: codes [pages][Hkv][ps][D], scale [pages][Hkv][ps / blk]."""
    s = np.asarray(scale).astype(np.int64)
    two = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return decode(codes) * np.repeat(two, codes.shape[2] // s.shape[2], axis=2)[..., None]


def quantise(cache, blk):
    """(codes, scale) of a whole cache, each block under its own scale."""
    pages, Hkv, ps, D = cache.shape
    blocks = np.asarray(cache, dtype=np.float64).reshape(pages, Hkv, ps // blk, blk, D)
    mag = np.where(np.isfinite(blocks), np.abs(blocks), 0.0).max((-1, -2))
    m, x = np.frexp(mag)
    e = np.maximum(np.where(mag > 0, x - 9 + (m > 0.875), LEAST), LEAST)
    codes = encode(np.ldexp(blocks, -e[..., None, None]))
    return codes.reshape(cache.shape), (e + 127).astype(np.uint8)


def norm(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def append(rows, codes, scale, table, prefix_len, active):
    """Copies of (codes, scale) of one cache with rows [B][Hkv][N][D] written where active [B][N]."""
    codes, scale = codes.copy(), scale.copy()
    ps = codes.shape[2]
    blk = ps // scale.shape[2]
    for b in range(rows.shape[0]):
        P = int(prefix_len[b])
        blocks = {}
        for t in np.flatnonzero(active[b]):
            blocks.setdefault((P + int(t)) // blk, []).append(int(t))
        for block, ts in blocks.items():
            page, r0 = int(table[b][block * blk // ps]), block * blk % ps
            held = max(0, P - block * blk)
            for h in range(rows.shape[1]):
                e = exponent(rows[b, h, ts])
                old = int(scale[page, h, r0 // blk]) - 127
                if held and old > e:
                    e = old
                if held and e > old:
                    keep = decode(codes[page, h, r0:r0 + held])
                    codes[page, h, r0:r0 + held] = encode(np.ldexp(keep, old - e))
                for t in ts:
                    codes[page, h, (P + t) % ps] = encode(np.ldexp(np.asarray(rows[b, h, t], np.float64), -e))
                scale[page, h, r0 // blk] = e + 127
    return codes, scale


def commit(codes, scale, table, prefix_len, accepted, accept_len):
    """Copies of (codes, scale) of one cache with every accepted path's rows at prefix_len + 1.. ."""
    was_c, was_s = codes, scale
    codes, scale = codes.copy(), scale.copy()
    ps = codes.shape[2]
    blk = ps // scale.shape[2]
    for b in range(len(prefix_len)):
        P, L = int(prefix_len[b]), int(accept_len[b])
        for h in range(codes.shape[1]):
            def at(r):
                return int(table[b][r // ps]), h, r % ps

            def of(r):
                p, _, k = at(r)
                return p, h, k // blk
            for block in range((P + 1) // blk, (P + L) // blk + 1 if L else 0):
                rows = range(block * blk, min(block * blk + blk, P + L + 1))
                src = [r if r <= P else P + int(accepted[b][r - P - 1]) for r in rows]
                s = max([int(was_s[of(block * blk)])] + [int(was_s[of(x)]) for x in src if x > P])
                for r, x in zip(rows, src):
                    codes[at(r)] = was_c[at(x)]
                    if int(was_s[of(x)]) != s:
                        codes[at(r)] = encode(np.ldexp(decode(was_c[at(x)]), int(was_s[of(x)]) - s))
                scale[of(block * blk)] = s
    return codes, scale
