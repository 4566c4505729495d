"""What fp32 attention over pages may be off by as a whole, and evaluations that must exceed it.

test_gpu_paged.py bounds each element by worst cases, which products of 11-bit inputs meet too.
Here the errors' root mean square over a head is bounded as that of independent roundings.  A sum of n
terms in fp32 rounds n partial sums by at most 2^-24 of what they hold, so its error is 2^-24 sqrt(n) of
that: for a score sqrt(D) Z, Z = max scale |q| |k_j| (norms) bounding every partial sum; 8 Z more for
the scale, the cap and what the exponential makes of them; sqrt(L) for the sums over L keys; 8 for the
exponential, the reciprocal and rescaling.  A weight's error moves the output by as much of p_j v_j, and
independent ones add up as the p_j v_j themselves do to the output:
  rms(error) <= 2^-24 ((sqrt(D) + 8) Z + sqrt(L) + 8) rms(output)
"""
import math

import numpy as np

import synth
from oracle import paged

# B, Hq, Hkv, D, page, prefixes, N, tree, softcap, window
CASES = [
    (2, 2, 2, 128, 16, [200, 2501], 1, False, 0.0, 0),      # one row a KV head
    (1, 2, 1, 64, 16, [271], 1, False, 0.0, 0),             # two
    (2, 4, 2, 128, 8, [764, 90], 2, True, 0.0, 0),          # four
    (1, 2, 2, 256, 32, [1300], 3, False, 0.0, 0),
    (1, 8, 1, 128, 16, [764], 1, False, 30.0, 0),           # eight
    (1, 8, 2, 64, 16, [900], 4, True, 0.0, 0),              # sixteen
    (2, 8, 2, 128, 16, [764, 200], 20, True, 0.0, 0),       # row tiles, clusters
    (1, 4, 1, 64, 16, [2501], 40, False, 0.0, 0),
    (1, 2, 1, 160, 16, [300], 30, False, 0.0, 0),
    (1, 2, 1, 256, 64, [500], 40, True, 20.0, 300),
    (45, 16, 8, 64, 16, [(13 * b) % 60 for b in range(45)], 9, False, 0.0, 0),   # row tiles, persistent grid
    (24, 16, 8, 128, 16, [(13 * b) % 60 for b in range(24)], 9, True, 0.0, 50),
]


def inputs(case):
    """q, k and v pages, table, parents (or None): every row of the pages holds numbers."""
    B, Hq, Hkv, D, ps, prefix, N, tree, _, _ = case
    g = synth.rng(5000 + D + N + max(prefix))
    width = (max(prefix) + N + ps - 1) // ps
    table = g.permutation(B * width).reshape(B, width).astype(np.int32)
    kc, vc = (synth.normal(g, (B * width, Hkv, ps, D), 1.0, False) for _ in range(2))
    par = np.stack([synth.random_parents(synth.rng(b), N, 12) for b in range(B)]).astype(np.int32) if tree else None
    return synth.normal(g, (B, Hq, N, D), 1.0, False), kc, vc, table, par


def reference(case, data):
    q, kc, vc, table, par = data
    return paged.attention(q, kc, vc, table, case[5], par, None, None, case[8], case[9])[0]


def worst(case, data, got, ref):
    """The largest rms(error) / bound over the heads."""
    q, kc, _, table, _ = data
    _, Hq, Hkv, D, ps, prefix, N, _, _, _ = case
    out = 0.0
    for b, P in enumerate(prefix):
        rows = [(table[b, r // ps], r % ps) for r in range(P + N)]
        norm = np.sqrt(np.max([np.sum(kc[p, :, r].astype(np.float64) ** 2, -1) for p, r in rows], 0))  # [Hkv]
        for h in range(Hq):
            Z = np.max(np.linalg.norm(q[b, h].astype(np.float64), axis=-1)) * norm[h * Hkv // Hq] / math.sqrt(D)
            bound = 2.0 ** -24 * ((math.sqrt(D) + 8) * Z + math.sqrt(P + N) + 8)
            err = np.sqrt(np.mean((got[b, h] - ref[b, h]) ** 2) / np.mean(ref[b, h] ** 2))
            out = max(out, err / bound)
    return out


def _bits(x, keep):
    """x rounded to `keep` explicit mantissa bits (10: TF32, 7: bf16)."""
    drop = 23 - keep
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + (1 << (drop - 1)) - 1 + ((u >> drop) & 1)) >> drop << drop
    return u.astype(np.uint32).view(np.float32)


def evaluate(case, data, qk=23, p=23, v=23):
    """The formula in fp32 on the host, queries and keys, weights, or values kept to fewer bits."""
    q, kc, vc, table, par = data
    B, Hq, Hkv, D, ps, prefix, N, _, cap, window = case
    f = np.float32
    rnd = lambda x, keep: x if keep == 23 else _bits(x, keep)  # noqa: E731
    out = np.zeros((B, Hq, N, D))
    for b, P in enumerate(prefix):
        at = np.arange(P + N)
        k, vv = (c[table[b][at // ps], :, at % ps] for c in (kc, vc))  # [L][Hkv][D]
        for i in range(N):
            path = list(range(i + 1))
            if par is not None:
                path = [i]
                while par[b, path[0]] >= 0:
                    path.insert(0, par[b, path[0]])
            where = len(path) - 1
            rows = [j for j in range(P) if not window or P + where - j < window]
            rows += [P + t for d, t in enumerate(path) if not window or where - d < window]
            for h in range(Hq):
                kk, x = rnd(k[rows, h * Hkv // Hq], qk), rnd(q[b, h, i], qk)
                z = (kk @ x) * f(1.0 / math.sqrt(D))
                if cap:
                    z = f(cap) * np.tanh(z / f(cap))
                w = np.exp(z - z.max())
                out[b, h, i] = (rnd(w, p) @ rnd(vv[rows, h * Hkv // Hq], v)) / w.sum(dtype=f)
    return out
