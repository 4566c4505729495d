"""GPU parity of the paged verification round against the oracle (64 bits): tv_rotary,
tv_append_kv_paged, tv_paged_attention, tv_commit_accepted_kv_paged, and a round of them.

Tolerances, per output element, u = eps / 2 of the type (2^-8 bf16, 2^-24 fp32):
  rotary  the pair's products in fp32: angle error below 2^-22 (a 2^-31 half turn and the
          sine's own error), four roundings: (|x| + |y|) A 2^-21; the frequencies, and the
          oracle's product of one with position p, hold a few 2^-53: p 2^-51 more; + u |out|
  attend  A = sum_j p_j |v_j|: a relative error e of every weight moves the output by at most
          2 e A.  e: the score's error, D products summed in fp32 at 2^-23 a step, on sums
          up to Z = max_j scale |q| . |k_j|, so 2 D 2^-23 Z; 2^-22 for the exponential; the cap's
          own error 2^-21 cap; L 2^-23 for the sums over L keys.  bf16 weights (rounded for
          the second product): 2^-8 A more.  Then u |out|.
"""
import math

import numpy as np
import pytest

import synth
import synth.workloads as W
from oracle import greedy, paged, rotary, tree, vocab

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import tree_speculative_decoding_masked_gb300 as tv  # noqa: E402
from gpu_util import dev, host, i32, to_dev  # noqa: E402

GARBAGE = (-7, 1 << 29, -(1 << 31), (1 << 31) - 1)


def _unit(bf16):
    return 2.0 ** -8 if bf16 else 2.0 ** -24


def _status():
    return torch.zeros(1, dtype=torch.int32, device=dev())


def _pages(g, B, Hkv, D, ps, lens, total, bf16, low=None, std=1.0):
    """Random pages and a table.  Rows [low_b, lens_b) of each sequence hold N(0, std), every
    other row NaN; table entries outside them hold garbage.  ``total`` rows are addressable."""
    width = (total + ps - 1) // ps + 2
    low = [0] * B if low is None else low
    need = [(max(lo, 0) // ps, (n + ps - 1) // ps) for lo, n in zip(low, lens)]
    count = sum(max(0, e - s) for s, e in need) + 3
    order = g.permutation(count)
    kc = np.full((count, Hkv, ps, D), np.nan, dtype=np.float32)
    vc = kc.copy()
    table = np.array([[GARBAGE[(b + p) % 4] for p in range(width)] for b in range(B)], dtype=np.int64).astype(np.int32)
    at = 0
    for b, (s, e) in enumerate(need):
        for p in range(s, e):
            table[b, p] = order[at]
            at += 1
        for r in range(max(low[b], 0), lens[b]):
            kc[table[b, r // ps], :, r % ps] = synth.normal(g, (Hkv, D), std, bf16)
            vc[table[b, r // ps], :, r % ps] = synth.normal(g, (Hkv, D), 1.0, bf16)
    return kc, vc, table


def _attend_check(g, B, Hq, Hkv, D, ps, prefix, N, *, parent=None, n_rows=None, softcap=0.0, window=0, bf16=True,
                  scale=None, std=1.0, workspace=None):
    act = [paged.active_rows(N, None if n_rows is None else n_rows[b], None if parent is None else parent[b])
           for b in range(B)]
    lens = [p + n if n else 0 for p, n in zip(prefix, act)]
    low = [p - window + 1 if window else 0 for p in prefix]
    # whole rows tables cover the declared rows; the trailing ones of a padded tree hold NaN
    kc, vc, table = _pages(g, B, Hkv, D, ps, lens, max(p + N for p in prefix), bf16, low, std)
    q = synth.normal(g, (B, Hq, N, D), std, bf16)
    out = torch.full((B, Hq, N, D), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
    st = _status()
    got = tv.paged_attention(to_dev(q, bf16), to_dev(kc, bf16), to_dev(vc, bf16), i32(table), i32(prefix),
                             parent=None if parent is None else i32(parent),
                             n_rows=None if n_rows is None else i32(n_rows), scale=0.0 if scale is None else scale,
                             softcap=softcap, window=window, out=out, workspace=workspace, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    got = host(got).astype(np.float64)
    ref, mass, big = paged.attention(q, kc, vc, table, prefix, parent, n_rows, scale, softcap, window)
    for b in range(B):
        assert np.all(got[b, :, act[b]:] == 7.0), "inactive rows were written"
        n = act[b]
        if n == 0:
            continue
        L = lens[b]
        e = 2 * D * 2.0 ** -23 * big[b, :, :n, None] + 2.0 ** -22 + L * 2.0 ** -23 + 2.0 ** -21 * softcap
        tol = (2 * e + (2.0 ** -8 if bf16 else 0)) * mass[b, :, :n] + _unit(bf16) * np.abs(ref[b, :, :n])
        err = np.abs(got[b, :, :n] - ref[b, :, :n])
        assert np.isfinite(got[b, :, :n]).all()
        worst = np.max(err / tol)
        assert worst <= 1.0, (b, worst)
    return got


# ---- attention

# B, Hq, Hkv, D, page, prefixes, N
TOKEN = [
    (1, 8, 2, 128, 16, [0], 1),          # the first token: itself alone
    (1, 8, 2, 128, 16, [1], 1),
    (2, 4, 4, 64, 8, [15, 16], 1),       # page ends
    (3, 32, 8, 128, 16, [700, 63, 64], 1),
    (1, 16, 1, 128, 32, [2500], 1),      # one KV head, many parts
    (5, 7, 7, 32, 64, [130, 0, 5, 129, 64], 1),
    (2, 6, 2, 96, 16, [40, 333], 1),     # G = 3, D = 96
    (2, 4, 2, 256, 128, [300, 127], 1),
    (1, 5, 5, 160, 8, [77], 1),
    (1, 24, 1, 64, 1024, [1500], 1),     # G = 24
]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", TOKEN)
def test_single_tokens(shape, bf16):
    B, Hq, Hkv, D, ps, prefix, N = shape
    _attend_check(synth.rng(900 + sum(shape[:5])), B, Hq, Hkv, D, ps, prefix, N, bf16=bf16)


CHUNK = [
    (1, 4, 2, 64, 16, [0], 2),
    (2, 4, 1, 128, 16, [37, 200], 5),    # 20 rows a head
    (2, 8, 2, 128, 16, [0, 129], 17),
    (1, 4, 4, 128, 8, [65], 64),         # G = 1
    (2, 8, 2, 128, 32, [100, 31], 45),
    (1, 8, 2, 64, 64, [64], 130),        # several row tiles
    (1, 6, 2, 128, 16, [3], 100),        # G = 3
    (1, 16, 1, 64, 128, [500], 33),      # G = 16
    (1, 24, 1, 128, 16, [50], 20),       # G = 24
    (1, 2, 1, 96, 16, [77], 140),
    (1, 2, 1, 32, 16, [20], 90),
    (1, 2, 1, 256, 16, [20], 70),
    (2, 4, 2, 128, 16, [1000, 3], 300),
]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", CHUNK)
def test_causal_chunks(shape, bf16):
    B, Hq, Hkv, D, ps, prefix, N = shape
    _attend_check(synth.rng(1000 + sum(shape[:5]) + N), B, Hq, Hkv, D, ps, prefix, N, bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", [
    (2, 8, 2, 128, 16, [100, 7], 3),
    (2, 8, 2, 128, 16, [300, 0], 40),
    (1, 4, 2, 64, 32, [70], 129),
    (1, 16, 2, 128, 64, [130], 70),
    (1, 4, 2, 96, 8, [33], 64),
    (1, 2, 2, 256, 16, [33], 50),
])
def test_trees(shape, bf16):
    B, Hq, Hkv, D, ps, prefix, N = shape
    g = synth.rng(1100 + sum(shape[:5]) + N)
    par, _ = W.trees(g, B, N, 6, 50)
    _attend_check(g, B, Hq, Hkv, D, ps, prefix, N, parent=par, bf16=bf16)


# row tile pairs enough for the persistent schedule, whose CTAs' ranges cross sequences, heads and pairs
PERSISTENT = [
    (3, 32, 32, 64, 16, [700, 10, 300], 40),
    (10, 32, 8, 128, 16, [0, 900, 5, 64, 63, 300, 1, 128, 17, 250], 20),
    (2, 32, 8, 128, 32, [3, 200], 300),
    (100, 3, 1, 96, 8, [(37 * b) % 90 for b in range(100)], 12),
    # few rows a head: 8, 16, 24 and 32 of them, and heads of 256
    (40, 16, 4, 128, 16, [(211 * b) % 1500 for b in range(40)], 2),
    (40, 16, 4, 128, 16, [(211 * b) % 1500 for b in range(40)], 4),
    (40, 16, 4, 64, 32, [(211 * b) % 1500 for b in range(40)], 6),
    (20, 32, 8, 128, 64, [(211 * b) % 900 for b in range(20)], 8),
    (20, 16, 8, 256, 16, [(211 * b) % 900 for b in range(20)], 4),
    (20, 16, 8, 256, 16, [(211 * b) % 900 for b in range(20)], 9),
]


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("tree_", [False, True])
@pytest.mark.parametrize("shape", PERSISTENT)
def test_persistent_schedule(shape, tree_, window):
    B, Hq, Hkv, D, ps, prefix, N = shape
    g = synth.rng(1170 + N + window)
    par, rows = None, [max(0, N - 3 * b) for b in range(B)]
    if tree_:
        par, _ = W.trees(g, B, N, 6, 50)
        rows = None
        for b in range(1, B):
            par[b, max(1, N - 2 * b):] = -1
    _attend_check(g, B, Hq, Hkv, D, ps, prefix, N, parent=par, n_rows=rows, window=window,
                  softcap=20.0 if window else 0.0)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N", [1, 11])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_persistent_schedule_of_every_head_size(D, N, bf16):
    g = synth.rng(1190 + D + N)
    B = 170 if D <= 64 else 80
    prefix = [(53 * b) % 150 for b in range(B)]
    _attend_check(g, B, 2, 1, D, 8, prefix, N, n_rows=[(b % (N + 1)) for b in range(B)], bf16=bf16, window=100,
                  softcap=15.0)


def test_equal_units_are_taken_whole():
    # 80 units of one length: one a CTA, uncut; a lone longer one changes that
    g = synth.rng(1195)
    for longest in (330, 1500):
        _attend_check(g, 10, 32, 8, 64, 64, [longest] + [330] * 9, 20)


@pytest.mark.parametrize("bf16", [True, False])
def test_deep_and_wide_trees(bf16):
    g = synth.rng(1150)
    N = 200
    par = np.stack([synth.chain_parents(N), synth.star_parents(N)]).astype(np.int32)
    _attend_check(g, 2, 4, 2, 64, 16, [90, 64], N, parent=par, bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N", [1, 9, 70])
def test_ragged_rows(bf16, N):
    # sequences with no rows, one row, all rows; padded trees; what is behind them stays
    g = synth.rng(1200 + N)
    rows = [0, 1, N, max(1, N // 2)]
    _attend_check(g, 4, 8, 2, 128, 16, [50, 0, 17, 128], N, n_rows=rows, bf16=bf16)
    par, _ = W.trees(g, 4, N, 5, 50)
    for b, n in enumerate(rows):
        par[b, max(1, n):] = -1
    _attend_check(g, 4, 8, 2, 128, 16, [50, 0, 17, 128], N, parent=par, bf16=bf16)
    _attend_check(g, 4, 8, 2, 128, 16, [50, 0, 17, 128], N, parent=par, n_rows=[min(r, 3) for r in rows], bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("window", [1, 2, 16, 33, 100, 5000])
@pytest.mark.parametrize("N", [1, 6, 80])
def test_windows(bf16, window, N):
    # rows behind every window are NaN and their table entries garbage
    g = synth.rng(1300 + N + window)
    _attend_check(g, 2, 8, 2, 64, 16, [250, 31], N, window=window, bf16=bf16)
    par, _ = W.trees(g, 2, N, 7, 50)
    _attend_check(g, 2, 8, 2, 64, 16, [250, 31], N, parent=par, window=window, bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("softcap", [0.5, 30.0])
@pytest.mark.parametrize("N", [1, 70])
def test_softcap(bf16, softcap, N):
    g = synth.rng(1400 + N)
    # scores far beyond the cap on both sides
    _attend_check(g, 2, 8, 2, 128, 16, [200, 9], N, softcap=softcap, bf16=bf16, std=2.0, scale=0.5)
    _attend_check(g, 2, 8, 2, 128, 16, [200, 9], N, softcap=softcap, window=40, bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N", [1, 90])
def test_growing_scores(bf16, N):
    # scores that climb along the keys move the running maximum again and again
    g = synth.rng(1500 + N)
    B, Hq, Hkv, D, ps, P = 1, 4, 1, 128, 16, 900
    kc, vc, table = _pages(g, B, Hkv, D, ps, [P + N], P + N, bf16)
    u = np.ones(D, dtype=np.float32)
    for r in range(P + N):
        kc[table[0, r // ps], 0, r % ps] = synth.round_to_bf16(
            (0.2 * kc[table[0, r // ps], 0, r % ps] + u * (6.0 * r / (P + N))).astype(np.float32))
    q = synth.round_to_bf16((np.abs(synth.normal(g, (B, Hq, N, D), 1.0, bf16))).astype(np.float32))
    got = host(tv.paged_attention(to_dev(q, bf16), to_dev(kc, bf16), to_dev(vc, bf16), i32(table), i32([P])))
    ref, mass, big = paged.attention(q, kc, vc, table, [P])
    e = 2 * D * 2.0 ** -23 * big[..., None] + 2.0 ** -22 + (P + N) * 2.0 ** -23
    tol = (2 * e + (2.0 ** -8 if bf16 else 0)) * mass + _unit(bf16) * np.abs(ref)
    assert np.max(np.abs(got - ref) / tol) <= 1.0


def test_many_sequences():
    # more sequences than a CTA has threads, most of them short
    g = synth.rng(1600)
    B = 600
    prefix = [int(x) for x in g.integers(0, 20, B)]
    prefix[599], prefix[300] = 400, 77
    _attend_check(g, B, 2, 1, 32, 8, prefix, 1, bf16=False)
    _attend_check(g, B, 2, 1, 64, 8, prefix, 1, bf16=True, n_rows=[int(x) for x in g.integers(0, 2, B)])


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N", [1, 70])
def test_one_workspace_many_shapes(bf16, N):
    # a workspace goes from call to call with nothing cleared in between
    dt = torch.bfloat16 if bf16 else torch.float32
    g = synth.rng(1700)
    n = max(tv.paged_attention_workspace_size(2, 8, 2, 128, N, 16, 64, dt),
            tv.paged_attention_workspace_size(1, 16, 1, 64, N, 16, 64, dt), 256)
    ws = torch.zeros(n, dtype=torch.uint8, device=dev())
    for _ in range(2):
        _attend_check(g, 2, 8, 2, 128, 16, [600, 90], N, bf16=bf16, workspace=ws)
        _attend_check(g, 1, 16, 1, 64, 16, [333], N, bf16=bf16, workspace=ws)


# more units than CTAs, short and long ones mixed, empty sequences between them: ranges of several
# pieces, cuts that move to a unit's edge and cuts that stay
MANY = [(60, 16, 4, 128, 16, 24, 40, True), (500, 4, 1, 64, 8, 1, 80, False), (9, 8, 2, 128, 64, 300, 30, False),
        (30, 8, 8, 64, 16, 33, 400, True), (420, 1, 1, 32, 8, 17, 60, False), (40, 8, 8, 128, 32, 3, 900, False),
        (3, 8, 4, 64, 128, 700, 700, False), (150, 16, 2, 256, 64, 1, 500, False), (25, 8, 4, 128, 8, 60, 2500, True)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,Hq,Hkv,D,ps,N,P,tree_", MANY)
def test_many_short_units(B, Hq, Hkv, D, ps, N, P, tree_, bf16):
    g = synth.rng(23)
    prefix = [int(x) for x in g.integers(0, P + 1, B)]
    prefix[:3] = [0, P, 1]
    n_rows = [int(x) for x in g.integers(0, N + 1, B)]
    n_rows[0] = N
    parent = np.stack([synth.random_parents(g, N, 8) for _ in range(B)]).astype(np.int32) if tree_ else None
    if tree_:
        for b in range(B):
            parent[b, max(n_rows[b], 1):] = -1
    window = 100 if N == 33 else 0
    first = _attend_check(synth.rng(24), B, Hq, Hkv, D, ps, prefix, N, parent=parent, n_rows=n_rows, window=window,
                          bf16=bf16)
    again = _attend_check(synth.rng(24), B, Hq, Hkv, D, ps, prefix, N, parent=parent, n_rows=n_rows, window=window,
                          bf16=bf16)
    assert np.array_equal(first, again)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N,Hkv,tree_", [(1, 2, False), (40, 2, True), (150, 2, False), (50, 40, True)])
def test_repeats_are_bit_equal_and_replay(bf16, N, Hkv, tree_):
    g = synth.rng(1800 + N)
    B, Hq, D, ps, prefix = 2, 4 * Hkv, 128, 16, [700, 321]
    kc, vc, table = _pages(g, B, Hkv, D, ps, [p + N for p in prefix], 900, bf16)
    par = W.trees(g, B, N, 6, 50)[0] if tree_ else None
    q = to_dev(synth.normal(g, (B, Hq, N, D), 1.0, bf16), bf16)
    kd, vd, td, pd = to_dev(kc, bf16), to_dev(vc, bf16), i32(table), i32(prefix)
    pard = None if par is None else i32(par)
    ws = torch.zeros(max(256, tv.paged_attention_workspace_size(B, Hq, Hkv, D, N, ps, table.shape[1], q.dtype)),
                     dtype=torch.uint8, device=dev())
    st, out = _status(), torch.zeros_like(q)

    def call():
        return tv.paged_attention(q, kd, vd, td, pd, parent=pard, out=out, workspace=ws, dev_status=st)
    first = call().clone()
    assert torch.equal(call(), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    # the lengths of the captured call live on the device: another round's prefix replays
    for lens in (prefix, [699, 5]):
        pd.copy_(i32(lens))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        again = out.clone()
        assert torch.equal(call(), again)
        assert torch.equal(again, first) == (lens == prefix)
    assert int(st.item()) == 0


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N", [1, 70])
def test_bad_pages_are_reported(bf16, N):
    # the kernels check every page number before they use it: nothing outside the pool is read,
    # and the other sequences' results stand
    g = synth.rng(1900 + N)
    B, Hq, Hkv, D, ps, prefix = 3, 8, 2, 64, 16, [100, 60, 90]
    kc, vc, table = _pages(g, B, Hkv, D, ps, [p + N for p in prefix], 200, bf16)
    q = synth.normal(g, (B, Hq, N, D), 1.0, bf16)
    ref = host(tv.paged_attention(to_dev(q, bf16), to_dev(kc, bf16), to_dev(vc, bf16), i32(table), i32(prefix)))
    for what in ("page", "low", "long", "negative", "rows"):
        t2, p2, rows = table.copy(), list(prefix), [N] * B
        if what == "page":
            t2[1, 2] = kc.shape[0]
        elif what == "low":
            t2[1, 0] = -1
        elif what == "long":
            p2[1] = table.shape[1] * ps
        elif what == "negative":
            p2[1] = -5
        else:
            rows[1] = N + 1
        st = _status()
        out = tv.paged_attention(to_dev(q, bf16), to_dev(kc, bf16), to_dev(vc, bf16), i32(t2), i32(p2),
                                 n_rows=i32(rows), dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == tv.TV_DEV_BAD_PAGE, what
        got = host(out)
        assert np.array_equal(got[0], ref[0]) and np.array_equal(got[2], ref[2]), what


def test_bad_trees_are_reported():
    g = synth.rng(1950)
    for N in (6, 70):
        kc, vc, table = _pages(g, 1, 2, 64, 16, [20 + N], 20 + N, True)
        q = to_dev(synth.normal(g, (1, 8, N, 64), 1.0, True), True)
        for at, p in ((0, 3), (4, 4), (4, 5), (4, -2), (3, -1)):
            par = synth.chain_parents(N)[None].astype(np.int32)
            par[0, at] = p
            st = _status()
            tv.paged_attention(q, to_dev(kc, True), to_dev(vc, True), i32(table), i32([20]), parent=i32(par),
                               dev_status=st)
            torch.cuda.synchronize()
            assert int(st.item()) == tv.TV_DEV_BAD_TREE, (N, at, p)


# ---- rotary and append

SCALINGS = [None, ("linear", 4.0), ("base", 8.0), ("banded", 8.0, 1.0, 4.0, 8192), ("yarn", 16.0, 4096, 32.0, 1.0)]


def _rot_tol(x, pos, rope, inter, bf16, ref):
    f, amp = rope
    half = len(f)
    mag = np.abs(x).astype(np.float64)
    pair = mag.copy()
    if inter:
        s = mag[..., 0:2 * half:2] + mag[..., 1:2 * half:2]
        pair[..., 0:2 * half:2], pair[..., 1:2 * half:2] = s, s
    else:
        s = mag[..., :half] + mag[..., half:2 * half]
        pair[..., :half], pair[..., half:2 * half] = s, s
    pair[..., 2 * half:] = 0
    far = 0 if pos is None else np.asarray(pos, dtype=np.float64)[:, None, :, None]
    return pair * amp * (2.0 ** -21 + far * 2.0 ** -51) + _unit(bf16) * np.abs(ref)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,H,N,D,rot,scaling", [
    (1, 32, 1, 128, 128, SCALINGS[0]),
    (2, 3, 7, 128, 64, SCALINGS[1]),
    (1, 2, 300, 64, 32, SCALINGS[2]),
    (3, 5, 11, 96, 96, SCALINGS[3]),
    (2, 40, 130, 128, 128, SCALINGS[4]),
    (2, 3, 5, 80, 20, SCALINGS[0]),      # 10 pairs: an element a thread
    (1, 2, 9, 7, 6, SCALINGS[1]),        # an odd head
    (1, 1, 3, 256, 0, None),             # nothing turns
    (1, 1, 3, 1024, 1024, None),
])
def test_rotary(B, H, N, D, rot, scaling, inter, bf16):
    g = synth.rng(2000 + D + rot + N)
    x = synth.normal(g, (B, H, N, D), 1.0, bf16)
    pos = g.integers(0, 1 << 20, (B, N)).astype(np.int32)
    pos[:, 0] = 0
    pos[-1, -1] = (1 << 31) - 1
    rope = tv.rotary_frequencies(rot, 500000.0, scaling=scaling) if rot else {
        "freq": torch.zeros(0, dtype=torch.int64, device=dev()), "amplitude": 1.0, "rot_dim": 0}
    ref_rope = rotary.frequencies(rot, 500000.0, scaling) if rot else (np.zeros(0), 1.0)
    ref = rotary.rotate(x, pos[:, None], *ref_rope, inter)
    tol = _rot_tol(x, pos, ref_rope, inter, bf16, ref)
    xd = to_dev(x, bf16)
    got = host(tv.rotary(xd, i32(pos), rope, interleaved=inter)).astype(np.float64)
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / np.maximum(tol, 1e-30))
    # token-major rows (a projection's output), rows with padding between them, a base
    big = torch.zeros((B, N, H, D + 8), dtype=xd.dtype, device=dev())
    big[..., :D] = xd.transpose(1, 2)
    base = i32(np.full(B, 5))
    got2 = tv.rotary(big[..., :D].transpose(1, 2), i32(pos - 5), rope, interleaved=inter, pos_base=base)
    neg = pos - 5 < 0  # rows that count as padding
    live = torch.from_numpy(~np.broadcast_to(neg[:, None], (B, H, N))).to(dev())
    assert torch.equal(got2[live], torch.from_numpy(got).to(got2)[live])
    # in place
    y = xd.clone()
    assert tv.rotary(y, i32(pos), rope, interleaved=inter, out=y) is y
    assert np.array_equal(host(y), host(tv.rotary(xd, i32(pos), rope, interleaved=inter)))


def test_rotary_skips_padding_and_unaligned_rows():
    g = synth.rng(2100)
    rope, ref_rope = tv.rotary_frequencies(32), rotary.frequencies(32)
    for bf16 in (True, False):
        x = synth.normal(g, (1, 2, 6, 32), 1.0, bf16)
        flat = torch.zeros(1 + x.size, dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
        flat[1:] = to_dev(x, bf16).reshape(-1)
        view = flat[1:].view(1, 2, 6, 32)  # rows one element off a 16-byte boundary
        pos = np.array([[3, -1, 7, -1, -5, 0]], dtype=np.int32)
        out = torch.full((1, 2, 6, 32), 9.0, dtype=view.dtype, device=dev())
        got = host(tv.rotary(view, i32(pos), rope, out=out)).astype(np.float64)
        ref = rotary.rotate(x, pos[:, None], *ref_rope)
        keep = pos[0] >= 0
        assert np.all(got[:, :, ~keep] == 9.0)
        tol = _rot_tol(x, pos, ref_rope, False, bf16, ref)
        assert np.all((np.abs(got - ref) <= tol)[:, :, keep])


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("B,Hq,Hkv,N,D,rot,ps,prefix,tree_", [
    (1, 8, 2, 1, 128, 128, 16, [0], False),
    (3, 4, 4, 5, 64, 32, 8, [7, 8, 123], False),
    (2, 6, 2, 37, 96, 96, 16, [100, 3], True),
    (2, 32, 8, 70, 128, 64, 64, [63, 500], True),
    (2, 2, 1, 9, 40, 20, 8, [5, 70], False),     # 10 pairs: an element a thread
    (1, 2, 1, 300, 256, 256, 1024, [1000], False),
])
def test_append(B, Hq, Hkv, N, D, rot, ps, prefix, tree_, with_q, bf16):
    g = synth.rng(2200 + D + N)
    par = W.trees(g, B, N, 5, 50)[0] if tree_ else None
    dep = rows = None
    if tree_:
        par[0, max(1, N // 2):] = -1  # a ragged batch
        dep = np.stack([np.where(np.arange(N) < tree.active_count(p), tree.depth(p), -1) for p in par]).astype(np.int32)
        prep = tv.tree_prep(i32(par), 0)
        assert np.array_equal(host(prep["depth"]), dep)
    else:
        rows = [max(0, N - 2 * b) for b in range(B)]
    kc, vc, table = _pages(g, B, Hkv, D, ps, [p + N for p in prefix], max(prefix) + N, bf16)
    qkv = synth.normal(g, (B, N, Hq + 2 * Hkv, D), 1.0, bf16)
    qkvd = to_dev(qkv, bf16).transpose(1, 2)
    qkv = qkv.transpose(0, 2, 1, 3)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    rope, (f, amp) = tv.rotary_frequencies(rot, scaling=SCALINGS[4]), rotary.frequencies(rot, scaling=SCALINGS[4])
    kd, vd, st = to_dev(kc, bf16), to_dev(vc, bf16), _status()
    qo = torch.full((B, Hq, N, D), 3.0, dtype=kd.dtype, device=dev())
    args = dict(depth=None if dep is None else i32(dep), n_rows=None if rows is None else i32(rows), rope=rope,
                dev_status=st, interleaved=True)
    if with_q:
        args.update(q=qkvd[:, :Hq], q_out=qo)
    got = tv.append_kv_paged(qkvd[:, Hq:Hq + Hkv], qkvd[:, Hq + Hkv:], kd, vd, i32(table), i32(prefix), **args)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (got is qo) == with_q
    kr, vr = paged.append(k, v, kc, vc, table, prefix, dep, rows, f, amp, True)
    assert np.array_equal(host(vd), vr.astype(np.float32), equal_nan=True)
    kg = host(kd).astype(np.float64)
    same = np.isnan(kr) | (kr == kc)
    assert np.array_equal(kg[same], kr[same], equal_nan=True)  # untouched rows, bit for bit
    bound = amp * 2.0 ** -21 * 2 * np.max(np.abs(k)) + _unit(bf16) * np.abs(kr)
    assert np.all(np.abs(kg - kr)[~same] <= bound[~same])
    if with_q:
        qg = host(qo).astype(np.float64)
        for b in range(B):
            n = tree.active_count(par[b]) if tree_ else rows[b]
            off = dep[b, :n] if tree_ else np.arange(n)
            ref = rotary.rotate(q[b, :, :n], (prefix[b] + off)[None], f, amp, True)
            tol = _rot_tol(q[b, :, :n], None, (f, amp), True, bf16, ref)
            assert np.all(np.abs(qg[b, :, :n] - ref) <= tol) and np.all(qg[b, :, n:] == 3.0)


def test_append_without_rotation_copies_bits():
    g = synth.rng(2300)
    kc, vc, table = _pages(g, 1, 2, 64, 8, [0], 30, True)
    bits = torch.from_numpy(g.integers(-32768, 32768, (1, 2, 20, 64)).astype(np.int16)).to(dev())  # NaNs among them
    kd, vd = to_dev(kc, True), to_dev(vc, True)
    table = np.arange(table.shape[1], dtype=np.int32)[None] % kc.shape[0]
    pool = torch.zeros((8, 2, 8, 64), dtype=torch.bfloat16, device=dev())
    pool_v = torch.zeros_like(pool)
    table = np.array([[5, 2, 7, 0]], dtype=np.int32)
    x = bits.view(torch.bfloat16)
    assert tv.append_kv_paged(x, x, pool, pool_v, i32(table), i32([3])) is None
    for r in range(20):
        at = pool.view(torch.int16)[table[0, (3 + r) // 8], :, (3 + r) % 8]
        assert torch.equal(at, bits[0, :, r])
    assert torch.equal(pool.view(torch.int16), pool_v.view(torch.int16))
    del kd, vd


def test_append_reports_bad_pages():
    g = synth.rng(2400)
    rope = tv.rotary_frequencies(64)
    x = to_dev(synth.normal(g, (2, 2, 4, 64), 1.0, True), True)
    for table, prefix in (([[0, 9], [1, 2]], [6, 6]), ([[0, -1], [1, 2]], [6, 6]), ([[0, 3], [1, 2]], [14, 6]),
                          ([[0, 3], [1, 2]], [-3, 6])):
        pool = torch.zeros((4, 2, 8, 64), dtype=torch.bfloat16, device=dev())
        pool_v, st = torch.zeros_like(pool), _status()
        tv.append_kv_paged(x, x, pool, pool_v, i32(table), i32(prefix), rope=rope, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == tv.TV_DEV_BAD_PAGE
        assert torch.equal(pool_v[1, :, 6:], x[1, :, :2]) and torch.equal(pool_v[2, :, :2], x[1, :, 2:])


# ---- commit

@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,Hkv,D,ps,prefix,N,lens", [
    (1, 8, 128, 16, [2048], 64, [5]),
    (3, 2, 64, 8, [0, 7, 100], 40, [0, 39, 12]),   # nothing, the whole chain, a path
    (2, 1, 256, 1024, [1000, 3], 1024, [1023, 700]),
    (70, 2, 40, 8, list(range(70)), 9, [b % 9 for b in range(70)]),
])
def test_commit(B, Hkv, D, ps, prefix, N, lens, bf16):
    g = synth.rng(2500 + N + D)
    kc, vc, table = _pages(g, B, Hkv, D, ps, [p + N for p in prefix], max(prefix) + N, bf16)
    acc = np.full((B, N), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        acc[b, :n] = np.sort(g.choice(np.arange(1, N), n, replace=False))
    kd, vd, st = to_dev(kc, bf16), to_dev(vc, bf16), _status()
    new = tv.commit_accepted_kv_paged(kd, vd, i32(table), i32(prefix), i32(acc), i32(lens), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert host(new).tolist() == [p + n + 1 for p, n in zip(prefix, lens)]
    assert np.array_equal(host(kd), paged.commit(kc, table, prefix, acc, lens), equal_nan=True)
    assert np.array_equal(host(vd), paged.commit(vc, table, prefix, acc, lens), equal_nan=True)


def test_commit_reports_bad_paths_and_pages():
    g = synth.rng(2600)
    for acc, n, t1, want in (([3, 2], 2, None, tv.TV_DEV_BAD_TREE), ([0, 2], 2, None, tv.TV_DEV_BAD_TREE),
                             ([-9, -8], 2, None, tv.TV_DEV_BAD_TREE), ([2, 8], 2, None, tv.TV_DEV_BAD_TREE),
                             ([2, 3], 8, None, tv.TV_DEV_BAD_TREE), ([2, 3], -1, None, tv.TV_DEV_BAD_TREE),
                             ([2, 6], 2, 99, tv.TV_DEV_BAD_PAGE), ([2, 6], 2, -1, tv.TV_DEV_BAD_PAGE)):
        kc, vc, table = _pages(g, 1, 2, 64, 8, [12], 12, False)
        if t1 is not None:
            table[0, 1] = t1
        path = np.full((1, 8), -1, dtype=np.int32)
        path[0, :2] = acc
        st = _status()
        tv.commit_accepted_kv_paged(to_dev(kc, False), to_dev(vc, False), i32(table), i32([4]), i32(path), i32([n]),
                                    dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == want, (acc, n, t1)


# ---- calls that the tests above do not make

@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N", [1, 60])
def test_no_active_rows_at_all(bf16, N):
    g = synth.rng(3000)
    _attend_check(g, 3, 8, 2, 64, 16, [0, 5, 200], N, n_rows=[0, 0, 0], bf16=bf16)
    pool = torch.full((4, 2, 16, 64), 2.0, dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
    x = torch.ones((1, 2, N, 64), dtype=pool.dtype, device=dev())
    st = _status()
    tv.append_kv_paged(x, x, pool, pool.clone(), i32([[0, 1, 2, 3, 0, 0]]), i32([3]), n_rows=i32([0]), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and bool((pool == 2.0).all())


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N", [1, 40])
def test_shared_and_repeated_pages(bf16, N):
    # two sequences with one prefix's pages, and a table that names a page twice
    g = synth.rng(3050 + N)
    B, Hq, Hkv, D, ps, P = 2, 8, 2, 64, 16, 64
    kc, vc, table = _pages(g, 1, Hkv, D, ps, [P + 5 * ps], P + 5 * ps, bf16)
    first = table[0, :9]
    shared = np.stack([np.concatenate([first[:4], first[4:7]]), np.concatenate([first[[0, 1, 0, 1]], first[6:9]])])
    shared = shared.astype(np.int32)
    q = synth.normal(g, (B, Hq, N, D), 1.0, bf16)
    got = host(tv.paged_attention(to_dev(q, bf16), to_dev(kc, bf16), to_dev(vc, bf16), i32(shared), i32([P, P])))
    ref, mass, big = paged.attention(q, kc, vc, shared, [P, P])
    e = 2 * D * 2.0 ** -23 * big[..., None] + 2.0 ** -22 + (P + N) * 2.0 ** -23
    tol = (2 * e + (2.0 ** -8 if bf16 else 0)) * mass + _unit(bf16) * np.abs(ref)
    assert np.max(np.abs(got - ref) / tol) <= 1.0


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N", [1, 100])
def test_pages_past_the_31st_bit(bf16, N):
    # a cache of more than 2^31 elements; the sequence sits in its last pages.  The calls on the last
    # pages give what they give on a small cache, bit for bit
    g = synth.rng(3100 + N)
    Hq, Hkv, D, ps, P = 16, 8, 128, 1024, 1500
    dt = torch.bfloat16 if bf16 else torch.float32
    big = (1 << 31) // (Hkv * ps * D) + 4
    gen = torch.Generator(device=dev())
    gen.manual_seed(5)
    small_k, small_v = (torch.randn((3, Hkv, ps, D), generator=gen, device=dev()).to(dt) for _ in range(2))
    qkv = torch.randn((1, N, Hq + 2 * Hkv, D), generator=gen, device=dev()).to(dt).transpose(1, 2)
    rope = tv.rotary_frequencies(D)
    acc = i32([sorted(g.choice(np.arange(1, max(N, 2)), min(N - 1, 12), replace=False)) + [-1] * (N - min(N - 1, 12))])
    results = []
    for pages, at in ((3, 0), (big, big - 3)):
        kc, vc = (torch.zeros((pages, Hkv, ps, D), dtype=dt, device=dev()) for _ in range(2))
        kc[at:at + 3], vc[at:at + 3] = small_k, small_v
        table, pre, st = i32([[at + 2, at]]), i32([P]), _status()
        q = tv.append_kv_paged(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kc, vc, table, pre, rope=rope, q=qkv[:, :Hq],
                               dev_status=st)
        out = tv.paged_attention(q, kc, vc, table, pre, dev_status=st)
        tv.commit_accepted_kv_paged(kc, vc, table, pre, acc, i32([min(N - 1, 12)]), dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        results.append((q, out, kc[at:at + 3].clone(), vc[at:at + 3].clone()))
        del kc, vc
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bf16", [True, False])
def test_two_calls_at_once(bf16):
    # two streams, a workspace each
    g = synth.rng(3150)
    dt = torch.bfloat16 if bf16 else torch.float32
    calls = []
    for N, Hkv in ((1, 2), (70, 2), (30, 32), (1, 40)):
        kc, vc, table = _pages(g, 3, Hkv, 64, 16, [600, 40, 333 + N], 700, bf16)
        args = (to_dev(synth.normal(g, (3, 2 * Hkv, N, 64), 1.0, bf16), bf16), to_dev(kc, bf16), to_dev(vc, bf16),
                i32(table), i32([600 - N, 40 - min(N, 30), 333]))
        n = tv.paged_attention_workspace_size(3, 2 * Hkv, Hkv, 64, N, 16, table.shape[1], dt)
        kw = dict(workspace=torch.zeros(max(n, 256), dtype=torch.uint8, device=dev()), n_rows=i32([N, min(N, 30), N]),
                  out=torch.zeros_like(args[0]))
        calls.append((args, kw, tv.paged_attention(*args, **dict(kw, out=torch.zeros_like(args[0]))).clone()))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for (args, kw, _), s in zip(calls, streams):
            with torch.cuda.stream(s):
                tv.paged_attention(*args, **kw)
    torch.cuda.synchronize()
    for _, kw, ref in calls:
        assert torch.equal(kw["out"], ref)


@pytest.mark.parametrize("bf16", [True, False])
def test_on_a_share_of_the_device(bf16):
    try:
        tv.set_sm_partition(0, 17)
        g = synth.rng(3200)
        for N in (1, 50):
            _attend_check(g, 12, 16, 8, 64, 16, [(97 * b) % 400 for b in range(12)], N, bf16=bf16)
    finally:
        tv.set_sm_partition(0, 0)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D,N,P", [(1, 1, 32, 65536, 3), (2, 1, 64, 20000, 777)])
def test_long_chunks(bf16, Hq, Hkv, D, N, P):
    # rows from all over a long chunk against 64-bit sums
    ps = 128
    dt = torch.bfloat16 if bf16 else torch.float32
    gen = torch.Generator(device=dev())
    gen.manual_seed(N)
    width = (P + N + ps - 1) // ps
    table = torch.randperm(width, generator=gen, device=dev()).int()[None]
    kc, vc = (torch.randn((width, Hkv, ps, D), generator=gen, device=dev()).to(dt) for _ in range(2))
    q = torch.randn((1, Hq, N, D), generator=gen, device=dev()).to(dt)
    st = _status()
    out = tv.paged_attention(q, kc, vc, table, i32([P]), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    k, v = (c[table[0].long()].permute(1, 0, 2, 3).reshape(Hkv, width * ps, D).double() for c in (kc, vc))
    for i in (0, 1, 62, 63, 64, 127, 128, 4095, 4096, 9999, N - 65, N - 64, N - 2, N - 1):
        for h in range(Hq):
            kk, vv, qi = k[0, :P + i + 1], v[0, :P + i + 1], q[0, h, i].double()
            z = kk @ qi / math.sqrt(D)
            p = torch.softmax(z, 0)
            ref, mass = p @ vv, p @ vv.abs()
            big = float((kk.abs() @ qi.abs()).max()) / math.sqrt(D)
            # sums over a long row: partial sums of tiles, so the keys of a tile and the tiles count
            e = 2 * D * 2.0 ** -23 * big + 2.0 ** -22 + (64 + (P + i) / 32) * 2.0 ** -23
            tol = (2 * e + (2.0 ** -8 if bf16 else 0)) * mass + _unit(bf16) * ref.abs()
            assert bool(((out[0, h, i].double() - ref).abs() <= tol).all()), (i, h)


def test_a_captured_round_replays():
    """append -> attention -> greedy verification -> commit, captured once; every replay is a round on
    the lengths that the last one left, and equals the same calls made eagerly."""
    g = synth.rng(3250)
    B, Hq, Hkv, D, ps, N, V = 2, 8, 2, 64, 16, 20, 50
    kc, vc, table = _pages(g, B, Hkv, D, ps, [300, 300], 300, True)
    rope, st = tv.rotary_frequencies(D), _status()
    par, tok = W.trees(g, B, N, 5, V)
    logits = to_dev(W.planted_logits(g, par, tok, V, False, prob=0.9), False)
    x = to_dev(synth.normal(g, (B, N, Hq + 2 * Hkv, D), 1.0, True), True).transpose(1, 2)
    pard, tokd, td = i32(par), i32(tok), i32(table)

    def setup():
        s = dict(k=to_dev(kc, True), v=to_dev(vc, True), lens=i32([7, 40]))
        s["q"] = torch.zeros((B, Hq, N, D), dtype=torch.bfloat16, device=dev())
        s["out"], s["new"] = torch.zeros_like(s["q"]), i32([0, 0])
        n = tv.paged_attention_workspace_size(B, Hq, Hkv, D, N, ps, table.shape[1], torch.bfloat16)
        s["ws"] = torch.zeros(max(n, 256), dtype=torch.uint8, device=dev())
        s["vws"] = torch.zeros(tv.verify_workspace_size(B, N, V, torch.float32, False), dtype=torch.uint8, device=dev())
        s["prep"] = {}
        return s

    def one(s):
        prep = tv.tree_prep(pard, 0, dev_status=st)
        tv.append_kv_paged(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], s["k"], s["v"], td, s["lens"], depth=prep["depth"],
                           rope=rope, q=x[:, :Hq], q_out=s["q"], dev_status=st)
        tv.paged_attention(s["q"], s["k"], s["v"], td, s["lens"], parent=pard, out=s["out"], workspace=s["ws"],
                           dev_status=st)
        res = tv.verify_greedy(logits, pard, tokd, workspace=s["vws"], dev_status=st)
        tv.commit_accepted_kv_paged(s["k"], s["v"], td, s["lens"], res["accepted_nodes"], res["accept_len"],
                                    new_len=s["new"], dev_status=st)
        s["lens"].copy_(s["new"])

    eager, captured, warm = setup(), setup(), setup()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one(warm)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(captured)
    for _ in range(4):
        one(eager)
        graph.replay()
        torch.cuda.synchronize()
        for key in ("lens", "q", "out"):
            assert torch.equal(eager[key], captured[key]), key
        for key in ("k", "v"):
            assert torch.equal(eager[key].view(torch.int16), captured[key].view(torch.int16)), key
    assert int(st.item()) == 0 and host(eager["lens"])[0] > 7 + 4


# ---- the calls together

@pytest.mark.parametrize("bf16", [True, False])
def test_rounds_over_pages(bf16):
    """Three rounds of prep -> append -> attention -> greedy verification -> commit on ragged
    sequences; after them the cache is that of the committed tokens laid end to end."""
    g = synth.rng(2700)
    B, Hq, Hkv, D, ps, N, V = 3, 8, 2, 64, 16, 24, 40
    prefix = [0, 15, 70]
    kc, vc, table = _pages(g, B, Hkv, D, ps, [p + 3 * N for p in prefix], max(prefix) + 3 * N, bf16)
    kd, vd, td = to_dev(kc, bf16), to_dev(vc, bf16), i32(table)
    pd = i32(prefix)
    rope, (f, amp) = tv.rotary_frequencies(D), rotary.frequencies(D)
    st = _status()
    for _ in range(3):
        par, tok = W.trees(g, B, N, 6, V)
        par[0, 20:] = -1
        logits = W.planted_logits(g, par, tok, V, False, prob=0.9)
        qkv = synth.normal(g, (B, N, Hq + 2 * Hkv, D), 1.0, bf16)
        x = to_dev(qkv, bf16).transpose(1, 2)
        pard = i32(par)
        prep = tv.tree_prep(pard, 0, dev_status=st)
        q = torch.zeros((B, Hq, N, D), dtype=kd.dtype, device=dev())
        tv.append_kv_paged(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kd, vd, td, pd, depth=prep["depth"], rope=rope,
                           q=x[:, :Hq], q_out=q, dev_status=st)
        out = tv.paged_attention(q, kd, vd, td, pd, parent=pard, dev_status=st)
        res = tv.verify_greedy(to_dev(logits, False), pard, i32(tok), dev_status=st)
        kt, vt = host(kd).astype(np.float64), host(vd).astype(np.float64)  # after the append
        new = tv.commit_accepted_kv_paged(kd, vd, td, pd, res["accepted_nodes"], res["accept_len"], dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        # the appended keys are the rotated rows
        for b in range(B):
            n = tree.active_count(par[b])
            dep = tree.depth(par[b])[:n]
            ref = rotary.rotate(qkv[b, :n, Hq:Hq + Hkv].transpose(1, 0, 2), (prefix[b] + dep)[None], f, amp)
            got = paged.rows_of(kt, table[b], prefix[b] + n)[:, prefix[b]:]
            assert np.all(np.abs(got - ref) <= 2.0 ** -21 * 16 + _unit(bf16) * np.abs(ref))
        qh = host(q).astype(np.float64)
        ref, mass, big = paged.attention(qh, kt, vt, table, prefix, par)
        err = np.abs(host(out).astype(np.float64) - ref)
        for b in range(B):
            n = tree.active_count(par[b])
            e = 2 * D * 2.0 ** -23 * big[b, :, :n, None] + 2.0 ** -22 + (prefix[b] + n) * 2.0 ** -23
            tol = (2 * e + (2.0 ** -8 if bf16 else 0)) * mass[b, :, :n] + _unit(bf16) * np.abs(ref[b, :, :n])
            assert np.all(err[b, :, :n] <= tol)
            _, _, am = vocab.vocab_stats(logits[b])
            path, _ = greedy.greedy_walk(par[b], tok[b], am)
            assert host(res["accepted_nodes"])[b, :len(path)].tolist() == path
            rows = [prefix[b] + t for t in [0] + path]
            want = paged.rows_of(kt, table[b], prefix[b] + n)[:, list(range(prefix[b])) + rows]
            prefix[b] += len(path) + 1
            assert np.array_equal(paged.rows_of(host(kd).astype(np.float64), table[b], prefix[b]), want)
        assert host(new).tolist() == prefix
        pd = new
