"""Pins of the paged-round oracle: rotary positions by hand-built values and by the property
that makes them position encodings, paged attention against the contiguous oracle, commit
against the contiguous one."""
import math

import numpy as np
import pytest

import synth
import synth.workloads as W
from oracle import attention, kvcommit, paged, rotary, tree


def _paginate(g, cache, ps, spare=3):
    """Contiguous [B][Hkv][S][D] -> random pages (unused rows NaN) and the table."""
    B, H, S, D = cache.shape
    width = (S + ps - 1) // ps
    order = g.permutation(B * width + spare)[:B * width].reshape(B, width).astype(np.int32)
    pages = np.full((B * width + spare, H, ps, D), np.nan)
    for b in range(B):
        for r in range(S):
            pages[order[b, r // ps], :, r % ps] = cache[b, :, r]
    return pages, order


def test_rotation_by_hand():
    f, amp = rotary.frequencies(4, 100.0)
    assert np.allclose(f, [1.0, 0.1]) and amp == 1.0
    y = rotary.rotate(np.array([1.0, 2.0, 3.0, 4.0, 5.0]), math.pi / 2, np.array([1.0, 2.0]))
    assert np.allclose(y, [-3.0, -2.0, 1.0, -4.0, 5.0])  # pairs (0, 2) by 90 and (1, 3) by 180 degrees
    y = rotary.rotate(np.array([1.0, 2.0, 3.0, 4.0, 5.0]), math.pi / 2, np.array([1.0, 2.0]), 2.0, True)
    assert np.allclose(y, [-4.0, 2.0, -6.0, -8.0, 5.0])  # pairs (0, 1) and (2, 3), amplitude 2


@pytest.mark.parametrize("inter", [False, True])
def test_products_depend_on_distance(inter):
    g = synth.rng(61)
    f, _ = rotary.frequencies(16)
    a, b = g.standard_normal(24), g.standard_normal(24)
    ref = rotary.rotate(a, 7, f, 1.0, inter) @ rotary.rotate(b, 3, f, 1.0, inter)
    far = rotary.rotate(a, 100007, f, 1.0, inter) @ rotary.rotate(b, 100003, f, 1.0, inter)
    assert abs(ref - far) < 1e-9


def test_scalings_at_their_ends():
    f, _ = rotary.frequencies(64, 10000.0)
    assert np.allclose(rotary.frequencies(64, 10000.0, ("linear", 4.0))[0], f / 4)
    s, _ = rotary.frequencies(64, 10000.0, ("base", 8.0))
    assert np.isclose(s[0], f[0]) and np.isclose(s[-1], f[-1] / 8)  # the slowest pair is slowed by the factor
    s, _ = rotary.frequencies(64, 10000.0, ("banded", 8.0, 1.0, 4.0, 8192))
    turns = 8192 * f / (2 * math.pi)
    assert np.allclose(s[turns > 4], f[turns > 4]) and np.allclose(s[turns < 1], f[turns < 1] / 8)
    s, amp = rotary.frequencies(64, 10000.0, ("yarn", 16.0, 4096, 32.0, 1.0))
    assert np.isclose(s[0], f[0]) and np.isclose(s[-1], f[-1] / 16) and np.isclose(amp, 0.1 * math.log(16) + 1)
    assert np.all(np.diff(s) < 0)


@pytest.mark.parametrize("ps", [8, 32])
def test_paged_attention_is_tree_attention(ps):
    g = synth.rng(62)
    B, Hq, Hkv, D, P, N = 2, 4, 2, 32, 21, 13
    par, _ = W.trees(g, B, N, 4, 50)
    q, k, v = W.qkv_host(g, B, Hq, Hkv, D, P, N, False)
    kp, table = _paginate(g, k, ps)
    vp = np.full_like(kp, np.nan)
    for b in range(B):
        for r in range(P + N):
            vp[table[b, r // ps], :, r % ps] = v[b, :, r]
    got, mass, _ = paged.attention(q, kp, vp, table, [P] * B, par)
    assert np.allclose(got, attention.tree_attention(q, k, v, par, P), atol=1e-12)
    assert np.all(mass >= np.abs(got) - 1e-12)


def test_causal_chunk_window_and_cap():
    g = synth.rng(63)
    Hq, D, P, N = 2, 32, 9, 6
    q, k, v = W.qkv_host(g, 1, Hq, 1, D, P, N, False)
    kp, table = _paginate(g, k, 8)
    vp = np.full_like(kp, np.nan)
    for r in range(P + N):
        vp[table[0, r // 8], :, r % 8] = v[0, :, r]
    got, _, _ = paged.attention(q, kp, vp, table, [P])
    for h in range(Hq):
        ref = attention.causal_attention(q[0, h], k[0, 0], v[0, 0], 1 / math.sqrt(D))
        assert np.allclose(got[0, h], ref, atol=1e-12)
    # window 1: every row sees itself alone
    got, _, _ = paged.attention(q, kp, vp, table, [P], window=1)
    assert np.allclose(got[0], np.broadcast_to(v[0, 0, P:], got[0].shape))
    # a chain tree is a causal chunk, with any window; a huge cap changes little, a tiny one evens the weights
    chain = synth.chain_parents(N)[None]
    for w in (0, 3, 8):
        a, _, _ = paged.attention(q, kp, vp, table, [P], window=w)
        b, _, _ = paged.attention(q, kp, vp, table, [P], parent=chain, window=w)
        assert np.allclose(a, b)
    a, _, _ = paged.attention(q, kp, vp, table, [P], softcap=1e6)
    b, _, _ = paged.attention(q, kp, vp, table, [P])
    assert np.allclose(a, b, atol=1e-9)
    a, _, _ = paged.attention(q, kp, vp, table, [P], softcap=1e-9)
    assert np.allclose(a[0, 0, 0], v[0, 0, :P + 1].mean(0))


def test_append_then_attend_and_commit():
    g = synth.rng(64)
    B, Hkv, D, P, N, ps = 2, 2, 32, 11, 9, 8
    par, tok = W.trees(g, B, N, 4, 50)
    _, k, v = W.qkv_host(g, B, 2, Hkv, D, P, N, False)
    empty_k, empty_v = k.copy(), v.copy()
    empty_k[:, :, P:], empty_v[:, :, P:] = 0, 0
    kp, table = _paginate(g, empty_k, ps)
    vp = np.zeros_like(kp)
    for b in range(B):
        for r in range(P + N):
            vp[table[b, r // ps], :, r % ps] = empty_v[b, :, r]
    dep = np.stack([tree.depth(par[b]) for b in range(B)])
    freq, _ = rotary.frequencies(D)
    ko, vo = paged.append(k[:, :, P:], v[:, :, P:], kp, vp, table, [P] * B, depth=dep, freq=freq)
    for b in range(B):
        assert np.allclose(paged.rows_of(vo, table[b], P + N), v[b])
        rows = paged.rows_of(ko, table[b], P + N)
        for t in range(N):
            assert np.allclose(rows[:, P + t], rotary.rotate(k[b, :, P + t], P + dep[b, t], freq))
    acc = np.full((B, N), -1, dtype=np.int32)
    path = tree.root_path(par[0], N - 1)[1:]
    acc[0, :len(path)] = path
    alen = [len(path), 0]
    ref, _ = kvcommit.commit_accepted(k, v, par, acc, alen, P)
    kp2, table2 = _paginate(g, k, ps)
    got = paged.commit(kp2, table2, [P] * B, acc, alen)
    for b in range(B):
        assert np.array_equal(paged.rows_of(got, table2[b], P + N), ref[b])
