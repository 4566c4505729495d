"""Rotary positions (oracle, float64).

What it restates
  * PTD §3.1: a node's position encoding follows |pi(v)|; the rotary encoding turns pair i
    of a query or key at position p by the angle p f_i (Su et al., "RoFormer", 2021).

Readings (not fixed by the pages)
  * The first R of a head's D elements form R / 2 pairs, (i, i + R / 2) or, interleaved,
    (2i, 2i + 1); the rest pass unchanged.
  * Frequencies f_i = base^(-2i / R), stretched for long contexts by one of: a common factor
    ("linear"), a larger base ("base"), a factor for the pairs that turn few times in the
    trained length ("banded"), or YaRN's ramp over the pair index with its amplitude.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot_dim: int, base: float = 10000.0, scaling=None):
    """(radians a position [rot_dim / 2], amplitude)."""
    out, amp = [], 1.0
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        if scaling is not None:
            kind, s = scaling[0], float(scaling[1])
            if kind == "linear":
                f = f / s
            elif kind == "base":
                f = (base * s ** (rot_dim / (rot_dim - 2.0))) ** (-2.0 * i / rot_dim)
            elif kind == "banded":
                lo, hi, length = scaling[2:]
                turns = length * f / (2 * math.pi)
                if turns < lo:
                    f = f / s
                elif turns <= hi:
                    w = (turns - lo) / (hi - lo)
                    f = w * f + (1 - w) * f / s
            elif kind == "yarn":
                length, fast, slow = scaling[2:]
                amp = 0.1 * math.log(s) + 1.0
                # the pair index whose pair turns `n` times in `length` positions
                first = max(math.floor(rot_dim * math.log(length / (fast * 2 * math.pi)) / (2 * math.log(base))), 0)
                last = min(math.ceil(rot_dim * math.log(length / (slow * 2 * math.pi)) / (2 * math.log(base))),
                           rot_dim - 1)
                w = min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
                f = (1 - w) * f + w * f / s
            else:
                raise ValueError(kind)
        out.append(f)
    return np.array(out, dtype=np.float64), amp


def rotate(x, pos, freq, amplitude: float = 1.0, interleaved: bool = False) -> np.ndarray:
    """x [..., D] at positions pos (broadcast over x's leading axes)."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    half = len(freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        # reduced before the product's rounding can matter: positions and turns stay below 2^53
        ang = np.asarray(pos, dtype=np.float64) * freq[i]
        c, s = np.cos(ang) * amplitude, np.sin(ang) * amplitude
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out
