"""One verification round over a paged cache (oracle, float64).

What it restates
  * The speculative-decoding blog's cache handling and PTD §3.1's tree mask, with the cache
    held in pages: cache row r of sequence b is row r mod page_size of page
    table[b][r // page_size], caches are [num_pages][Hkv][page_size][D].

Readings (not fixed by the pages)
  * Sequence b has prefix_len[b] committed rows and new rows at prefix_len[b] + t; new row i
    sees the committed rows and new rows t <= i (a chunk) or pi(i) (a tree), less those
    `window` or more positions back, where new row t sits at position prefix_len[b] + t, or
    prefix_len[b] + depth(t) in a tree.
  * softcap: z -> softcap tanh(z / softcap) before the softmax.
  * Rows from n_rows[b] on, and padding rows of a tree, are inactive.
"""
from __future__ import annotations

import math

import numpy as np

from . import rotary
from .tree import is_padding, root_path


def active_rows(n, n_rows_b, parent_b):
    n = n if n_rows_b is None else int(n_rows_b)
    if parent_b is not None:
        for t in range(1, n):
            if is_padding(parent_b, t):
                return t
    return n


def rows_of(cache, table_b, length, first=0):
    """[Hkv][length][D] of one sequence; rows before `first` are not looked up (NaN)."""
    ps = cache.shape[2]
    out = np.full((cache.shape[1], length, cache.shape[3]), np.nan)
    for r in range(first, length):
        out[:, r] = cache[table_b[r // ps], :, r % ps]
    return out


def attention(q, k_cache, v_cache, table, prefix_len, parent=None, n_rows=None, scale=None, softcap=0.0, window=0):
    """(out [B][Hq][N][D], sum_j p_j |v_j| likewise, max_j sum_d |q_d k_jd| scale [B][Hq][N]); inactive rows 0."""
    q = np.asarray(q, dtype=np.float64)
    B, Hq, N, D = q.shape
    G = Hq // k_cache.shape[1]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out, mass, big = np.zeros_like(q), np.zeros_like(q), np.zeros((B, Hq, N))
    for b in range(B):
        P = int(prefix_len[b])
        par = None if parent is None else parent[b]
        n = active_rows(N, None if n_rows is None else n_rows[b], par)
        if n == 0:
            continue
        low = max(0, P - window + 1) if window else 0  # behind it no row sees anything
        k, v = rows_of(k_cache, table[b], P + n, low), rows_of(v_cache, table[b], P + n, low)
        for i in range(n):
            path = list(range(i + 1)) if par is None else root_path(par, i)
            where = len(path) - 1  # position - P
            rows = [j for j in range(P) if not window or P + where - j < window]
            rows += [P + t for d, t in enumerate(path) if not window or where - d < window]
            for h in range(Hq):
                kk, vv = k[h // G, rows], v[h // G, rows]
                z = kk @ q[b, h, i] * scale
                big[b, h, i] = np.max(np.abs(kk) @ np.abs(q[b, h, i])) * scale
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                p = np.exp(z - z.max())
                p /= p.sum()
                out[b, h, i], mass[b, h, i] = p @ vv, p @ np.abs(vv)
    return out, mass, big


def append(k, v, k_cache, v_cache, table, prefix_len, depth=None, n_rows=None, freq=None, amplitude=1.0,
           interleaved=False):
    """Copies of the caches with the new rows written (float64)."""
    ko, vo = np.array(k_cache, dtype=np.float64), np.array(v_cache, dtype=np.float64)
    B, _, N, _ = k.shape
    ps = k_cache.shape[2]
    for b in range(B):
        for t in range(N if n_rows is None else int(n_rows[b])):
            off = t if depth is None else int(depth[b][t])
            if off < 0:
                continue
            r = int(prefix_len[b]) + t
            row = np.asarray(k[b, :, t], dtype=np.float64)
            if freq is not None:
                row = rotary.rotate(row, int(prefix_len[b]) + off, freq, amplitude, interleaved)
            ko[table[b][r // ps], :, r % ps] = row
            vo[table[b][r // ps], :, r % ps] = v[b, :, t]
    return ko, vo


def commit(cache, table, prefix_len, accepted, accept_len):
    """Copy of the cache with every accepted path's rows at prefix_len + 1.. ."""
    out, ps = np.array(cache, copy=True), cache.shape[2]
    for b in range(len(prefix_len)):
        P = int(prefix_len[b])
        for k in range(1, int(accept_len[b]) + 1):
            i, j = P + int(accepted[b][k - 1]), P + k
            out[table[b][j // ps], :, j % ps] = cache[table[b][i // ps], :, i % ps]
    return out
