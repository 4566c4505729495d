"""Pins of the 8-bit cache oracle: the code table against torch's type, rounding against brute force,
scales against their definition, and what an append and a commit keep."""
import numpy as np
import pytest

import synth
from oracle import paged_q8 as q8

torch = pytest.importorskip("torch")


def test_codes_are_the_types():
    c = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(q8.decode(c), ref, equal_nan=True)


def test_encode_takes_the_nearest_and_even_on_ties():
    finite = q8.decode(np.arange(127, dtype=np.uint8))
    mids = (finite[1:] + finite[:-1]) / 2
    g = synth.rng(1)
    x = np.concatenate((finite, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9), g.uniform(0, 448, 5000)))
    x = np.concatenate((x, -x))
    codes = q8.encode(x)
    err = np.abs(q8.decode(codes) - x)
    best = np.min(np.abs(np.abs(x)[:, None] - finite[None]), axis=1)
    assert np.array_equal(err, best)
    assert np.all(q8.encode(mids) % 2 == 0)
    assert np.all(np.isnan(q8.decode(q8.encode([np.inf, -np.inf, np.nan]))))
    # torch rounds alike
    t = torch.from_numpy(x).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    exact = x == x.astype(np.float32)
    assert np.array_equal(t[exact], q8.decode(codes)[exact])


def test_exponents():
    for top, e in ((448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (0.0, -117), (1e-40, -117), (3.38e38, 120)):
        assert q8.exponent([0.0, -top, np.nan, np.inf]) == e
    cache = synth.rng(2).standard_normal((3, 2, 16, 32)) * 10.0 ** synth.rng(3).integers(-6, 6, (3, 2, 16, 1))
    for blk in (1, 4, 16):
        codes, scale = q8.quantise(cache, blk)
        for p in range(3):
            for k in range(16 // blk):
                assert int(scale[p, 1, k]) - 127 == q8.exponent(cache[p, 1, k * blk:(k + 1) * blk])
        x, two = q8.numbers(codes, scale), np.repeat(np.ldexp(1.0, scale.astype(int) - 127), blk, 2)[..., None]
        assert np.all(np.abs(x - cache) <= np.maximum(np.abs(cache) * 2.0 ** -4, two * 2.0 ** -10))


def test_append_grows_a_scale_and_keeps_the_numbers():
    g = synth.rng(4)
    codes, scale = np.full((3, 1, 16, 32), 127, np.uint8), np.full((3, 1, 2), 255, np.uint8)
    table = np.array([[2, 0]])
    small = g.standard_normal((1, 1, 5, 32))
    c1, s1 = q8.append(small, codes, scale, table, [0], np.ones((1, 5), bool))
    before = q8.numbers(c1, s1)[2, 0, :5]
    c2, s2 = q8.append(small[:, :, :6] * 64, c1, s1, table, [5], np.ones((1, 5), bool))
    assert s2[2, 0, 0] > s1[2, 0, 0]
    after = q8.numbers(c2, s2)[2, 0, :5]
    step = 2.0 ** (int(s2[2, 0, 0]) - 127 - 9)
    assert np.all(np.abs(after - before) <= step / 2) and np.mean(after == before) > 0.5
    # a smaller row leaves the scale, a fresh block takes its own
    c3, s3 = q8.append(small / 64, c2, s2, table, [7], np.array([[True, True, False, False, False]]))
    assert s3[2, 0, 0] == s2[2, 0, 0] and s3[2, 0, 1] < s2[2, 0, 1]
    assert np.array_equal(c3[2, 0, :7], c2[2, 0, :7]) and np.array_equal(c3[0], codes[0])


def test_commit_moves_numbers():
    g = synth.rng(5)
    cache = g.standard_normal((4, 2, 8, 32)) * 2.0 ** g.integers(-3, 4, (4, 2, 8, 1))
    codes, scale = q8.quantise(cache, 4)
    table = np.array([[3, 1, 0, 2]])
    P, path = 5, [2, 6, 11, 13]
    c, s = q8.commit(codes, scale, table, [P], [path], [4])
    was, now = q8.numbers(codes, scale), q8.numbers(c, s)
    rows = [(table[0][r // 8], r % 8) for r in range(32)]
    for k, a in enumerate(path):
        src, dst = rows[P + a], rows[P + k + 1]
        step = np.ldexp(1.0, s[dst[0], :, dst[1] // 4].astype(int) - 136)[:, None]
        assert np.all(np.abs(now[dst[0], :, dst[1]] - was[src[0], :, src[1]]) <= step / 2)
    for r in range(P + 1):
        p, k = rows[r]
        step = np.ldexp(1.0, s[p, :, k // 4].astype(int) - 136)[:, None]
        assert np.all(np.abs(now[p, :, k] - was[p, :, k]) <= step / 2)
    for r in range(P + 5, 32):
        assert np.array_equal(c[rows[r][0], :, rows[r][1]], codes[rows[r][0], :, rows[r][1]])


def test_norm():
    x = synth.rng(6).standard_normal((2, 3, 8))
    y = q8.norm(x, np.full(8, 2.0), 0.0)
    assert np.allclose(np.mean(y * y, -1), 4.0)
