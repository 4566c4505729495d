"""GPU parity of attention over 8-bit pages whose value blocks have scales far apart: blocks of zeros (the append gives
them 2^-117), values near both ends of the scales, and mixtures, against the oracle (64 bits).

Tolerance as in test_gpu_paged_q8.py, with two terms more for bf16 rows, u = 2^-8:
  z + e   a score and a value's exponent (|z| log2 e + 127 < 2^8) meet in fp32 and their sum less a reference is an
          exponent of two: two roundings of 2^-17 each, a weight is off by ln 2 * 2^-16 < 2^-16 of itself, numerator
          and sum alike
  fp16    a weight times its block's scale is held in fp16, the row's largest at 2^7 or above and the least number
          2^-24: one may be off by 2^-25 / 2^7 of the largest besides its own rounding, times the block's codes
"""
import math

import numpy as np
import pytest

import synth
import synth.workloads as W
from oracle import paged, paged_q8 as q8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import tree_speculative_decoding_masked_gb300 as tv  # noqa: E402
from gpu_util import dev, host, i32, to_dev  # noqa: E402
from test_gpu_paged import _pages, _status, _unit  # noqa: E402


def _zeros(where):
    """Factor of value row r of a sequence of L rows, by name."""
    def factor(r, L):
        if where == "all":
            return 0.0
        if where == "middle":
            return 0.0 if L // 3 <= r < 2 * L // 3 else 1.0
        if where == "last":
            return 0.0 if r >= L // 2 else 1.0
        if where == "every other 16":
            return float(r // 16 % 2)
        if where == "beside 2^30":
            return (0.0, 2.0 ** 30, 1.0)[r // 16 % 3]
        if where == "2^-90 to 2^90":
            return 2.0 ** (-90, -45, 0, 45, 90)[r // 16 % 5]
        return 0.0 if r < int(where) else 1.0
    return factor


def _far_check(g, B, Hq, Hkv, D, ps, prefix, N, factor, *, blk, bf16, parent=None, n_rows=None, window=0, lean=0.0,
               softcap=0.0):
    act = [paged.active_rows(N, None if n_rows is None else n_rows[b], None if parent is None else parent[b])
           for b in range(B)]
    lens = [p + n if n else 0 for p, n in zip(prefix, act)]
    low = [max(0, p - window + 1) if window else 0 for p in prefix]
    kc, vc, table = _pages(g, B, Hkv, D, ps, lens, max(p + N for p in prefix), False, low, 1.0)
    q = synth.normal(g, (B, Hq, N, D), 1.0, bf16)
    vc = vc.astype(np.float64)
    for b in range(B):
        for r in range(low[b], lens[b]):
            f = factor(r, lens[b])
            vc[table[b, r // ps], :, r % ps] *= f
            if f == 0.0 and lean:  # the rows of zeros draw the queries, or repel them
                kc[table[b, r // ps], :, r % ps] += lean * np.sign(q[0, 0, 0])
    kc, ks = q8.quantise(kc, blk)
    vc, vs = q8.quantise(vc, blk)
    st = _status()
    out = torch.full((B, Hq, N, D), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())

    def call():
        return tv.paged_attention(to_dev(q, bf16), torch.from_numpy(kc).to(dev()).view(torch.float8_e4m3fn),
                                  torch.from_numpy(vc).to(dev()).view(torch.float8_e4m3fn), i32(table), i32(prefix),
                                  parent=None if parent is None else i32(parent),
                                  n_rows=None if n_rows is None else i32(n_rows), softcap=softcap, window=window, out=out,
                                  dev_status=st, k_scale=torch.from_numpy(ks).to(dev()),
                                  v_scale=torch.from_numpy(vs).to(dev())).clone()
    got = call()
    assert torch.equal(call(), got) and int(st.item()) == 0
    got = host(got).astype(np.float64)
    for b in range(B):
        assert np.all(got[b, :, act[b]:] == 7.0), "inactive rows were written"
    _compare(got, q, kc, ks, vc, vs, table, prefix, act, lens, low, parent, n_rows, bf16, window, softcap)
    return got


def _compare(got, q, kc, ks, vc, vs, table, prefix, act, lens, low, parent, n_rows, bf16, window=0, softcap=0.0):
    B, Hq, _, D = q.shape
    Hkv, ps = kc.shape[1], kc.shape[2]
    with np.errstate(all="ignore"):
        k, v = q8.numbers(kc, ks), q8.numbers(vc, vs)
        codes = np.abs(q8.decode(vc))
        ref, mass, big = paged.attention(q, k, v, table, prefix, parent, n_rows, None, softcap, window)
    for b in range(B):
        n, L = act[b], lens[b]
        if n == 0:
            continue
        rows = [(table[b, r // ps], r % ps) for r in range(low[b], L)]
        e = 2 * D * 2.0 ** -23 * big[b, :, :n, None] + 2.0 ** -22 + L * 2.0 ** -23 + 2.0 ** -21 * softcap
        tol = 0.0
        if bf16:
            norm = np.repeat(np.max([np.abs(k[p, :, r]).sum(-1) for p, r in rows], 0), Hq // Hkv)
            e = e + 2.0 ** -16 + 2.0 ** -17 / math.sqrt(D) * (np.abs(q[b, :, :n]).max(-1) * norm[:, None])[..., None]
            top = np.max([2.0 ** (vs[p, :, r // (ps // vs.shape[2])].astype(float) - 127) for p, r in rows], 0)
            tol = (2.0 ** -32 * np.repeat(top[:, None] * np.sum([codes[p, :, r] for p, r in rows], 0), Hq // Hkv, 0))[:, None]
        tol = tol + (2 * e + (2.0 ** -8 if bf16 else 0)) * mass[b, :, :n] + _unit(bf16) * np.abs(ref[b, :, :n])
        assert np.isfinite(got[b, :, :n]).all(), b
        worst = np.max(np.abs(got[b, :, :n] - ref[b, :, :n]) / np.maximum(tol, 1e-300))
        assert worst <= 1.0, (b, worst)


WHERE = ["16", "64", "300", "all", "middle", "last", "every other 16", "beside 2^30", "2^-90 to 2^90"]


# one sequence: clusters, or pieces of a unit
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("blk", [1, 16])
@pytest.mark.parametrize("N", [1, 4, 8, 90])
@pytest.mark.parametrize("where", WHERE)
def test_attend_zero_values(where, N, blk, bf16):
    for lean in (0.0, 0.5, -0.5) if N < 90 else (0.5,):
        _far_check(synth.rng(7000 + N + blk), 1, 8, 2, 128, 16, [1100], N, _zeros(where), blk=blk, bf16=bf16, lean=lean)


@pytest.mark.parametrize("D,ps", [(32, 8), (64, 64), (96, 16), (160, 16), (256, 32)])
@pytest.mark.parametrize("N", [1, 6, 40])
@pytest.mark.parametrize("where", ["64", "middle", "beside 2^30"])
def test_attend_zero_values_of_every_head_size(where, N, D, ps):
    _far_check(synth.rng(7100 + N + D), 2, 4, 2, D, ps, [700, 33], N, _zeros(where), blk=min(ps, 16), bf16=True)
    par, _ = W.trees(synth.rng(7101), 2, N, 5, 50)
    _far_check(synth.rng(7102 + N + D), 2, 4, 2, D, ps, [300, 5], N, _zeros(where), blk=4, bf16=True, parent=par,
               softcap=20.0)


# many units on the persistent grids: whole ones, and cut ones whose parts hold zeros alone
@pytest.mark.parametrize("where", ["16", "middle", "beside 2^30"])
@pytest.mark.parametrize("B,Hq,Hkv,D,N,P,blk", [(40, 8, 4, 128, 1, 1500, 16), (40, 16, 4, 128, 4, 900, 16),
                                                (40, 16, 4, 128, 4, 600, 2), (12, 32, 8, 64, 4, 700, 16),
                                                (10, 16, 8, 128, 40, 900, 16), (3, 32, 16, 64, 64, 1400, 2)])
def test_attend_zero_values_persistent(B, Hq, Hkv, D, N, P, blk, where):
    prefix = [(211 * b + P) % (P + 1) for b in range(B)]
    rows = [N - b % 2 * (N // 3) for b in range(B)]
    _far_check(synth.rng(7200 + N + D), B, Hq, Hkv, D, 16, prefix, N, _zeros(where), blk=blk, bf16=True, n_rows=rows)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N", [1, 4, 90])
@pytest.mark.parametrize("window", [40, 600])
def test_attend_zero_values_behind_a_window(window, N, bf16):
    # a far block within the window of some rows and behind that of others
    for where in ("300", "last", "every other 16"):
        _far_check(synth.rng(7300 + N), 1, 8, 2, 128, 16, [900], N, _zeros(where), blk=16, bf16=bf16, window=window)


@pytest.mark.parametrize("softcap", [20.0, 1000.0])
@pytest.mark.parametrize("blk", [1, 16])
@pytest.mark.parametrize("N", [1, 4, 70])
def test_attend_zero_values_under_a_cap(N, blk, softcap):
    for where in ("64", "beside 2^30", "2^-90 to 2^90"):
        _far_check(synth.rng(7350 + N), 1, 8, 2, 128, 16, [500], N, _zeros(where), blk=blk, bf16=True, softcap=softcap)


def _bytes_check(N, blk, draw, prefix=700):
    """All scales of V's needed blocks as `draw` gives them, under codes of any size."""
    g = synth.rng(7400 + N + blk)
    kc, vc, table = _pages(g, 1, 2, 128, 16, [prefix + N], prefix + N, False, [0], 1.0)
    kc, ks = q8.quantise(kc, blk)
    vc, vs = q8.quantise(vc, blk)
    vs = draw(g, vs.shape).astype(np.uint8)
    q = synth.normal(g, (1, 8, N, 128), 1.0, True)
    got = host(tv.paged_attention(to_dev(q, True), torch.from_numpy(kc).to(dev()).view(torch.float8_e4m3fn),
                                  torch.from_numpy(vc).to(dev()).view(torch.float8_e4m3fn), i32(table), i32([prefix]),
                                  k_scale=torch.from_numpy(ks).to(dev()), v_scale=torch.from_numpy(vs).to(dev())))
    _compare(got.astype(np.float64), q, kc, ks, vc, vs, table, [prefix], [N], [prefix + N], [0], None, None, True)


@pytest.mark.parametrize("blk", [1, 16])
@pytest.mark.parametrize("N", [1, 4, 90])
def test_attend_values_of_the_least_scale(N, blk):
    _bytes_check(N, blk, lambda g, n: np.full(n, 10))
    _bytes_check(N, blk, lambda g, n: g.choice([10, 127], n))
    _bytes_check(N, blk, lambda g, n: g.choice([10, 86, 87, 167, 168], n))


# codes up to 448 under 2^119 stay below 2^128, in bf16 too
@pytest.mark.parametrize("blk", [1, 16])
@pytest.mark.parametrize("N", [1, 4, 90])
def test_attend_values_of_the_largest_numbers(N, blk):
    _bytes_check(N, blk, lambda g, n: np.full(n, 119 + 127))
    _bytes_check(N, blk, lambda g, n: g.choice([10, 100, 200, 246], n))


@pytest.mark.parametrize("blk", [1, 16])
@pytest.mark.parametrize("N", [1, 4, 90])
def test_attend_values_of_the_largest_scale(N, blk):
    # byte 254 with codes of 1 at most: beside others each key counts once, and alone its number is the answer
    g = synth.rng(7500 + N + blk)
    P = 200
    kc, vc, table = _pages(g, 1, 2, 64, 16, [P + N], P + N, False, [0], 1.0)
    kc, ks = q8.quantise(kc, blk)
    vc = q8.encode(np.where(np.isnan(vc), np.nan, np.clip(vc / 8, -1, 1)))
    q = synth.normal(g, (1, 4, N, 64), 1.0, True)
    for choice in ([254], [254, 127], [254, 10], [253]):
        vs = g.choice(choice, ks.shape).astype(np.uint8)
        got = host(tv.paged_attention(to_dev(q, True), torch.from_numpy(kc).to(dev()).view(torch.float8_e4m3fn),
                                      torch.from_numpy(vc).to(dev()).view(torch.float8_e4m3fn), i32(table), i32([P]),
                                      k_scale=torch.from_numpy(ks).to(dev()), v_scale=torch.from_numpy(vs).to(dev())))
        _compare(got.astype(np.float64), q, kc, ks, vc, vs, table, [P], [N], [P + N], [0], None, None, True)


@pytest.mark.parametrize("N", [1, 4, 70])
def test_attend_nan_query_over_zero_values(N):
    g = synth.rng(7600)
    for B, Hkv in ((2, 2), (40, 8)):
        lens = [200 + N] * B
        kc, vc, table = _pages(g, B, Hkv, 64, 16, lens, 200 + N, False, [0] * B, 1.0)
        vc[table[:, :6]] = 0.0
        kc, ks = q8.quantise(kc, 16)
        vc, vs = q8.quantise(vc, 16)
        q = to_dev(synth.normal(g, (B, 4 * Hkv, N, 64), 1.0, True), True)
        args = [torch.from_numpy(x).to(dev()).view(torch.float8_e4m3fn) for x in (kc, vc)] + [i32(table), i32([200] * B)]
        s = dict(k_scale=torch.from_numpy(ks).to(dev()), v_scale=torch.from_numpy(vs).to(dev()))
        ref = tv.paged_attention(q, *args, **s)
        assert torch.isfinite(ref).all()
        q2 = q.clone()
        q2[1, 3, N - 1, 17] = float("nan")
        got = tv.paged_attention(q2, *args, **s)
        assert torch.isnan(got[1, 3, N - 1]).all()
        got[1, 3, N - 1] = ref[1, 3, N - 1]
        assert torch.equal(got, ref)


@pytest.mark.parametrize("N", [1, 4, 90])
def test_appended_zero_values_are_attended(N):
    # values of zeros through the append, as a model with a dead head writes them, and ordinary ones behind
    g = synth.rng(7700 + N)
    Hkv, D, P = 2, 128, 512
    pages = (P + N + 15) // 16
    kc, vc = (torch.zeros(pages, Hkv, 16, D, dtype=torch.uint8, device=dev()).view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(pages, Hkv, 1, dtype=torch.uint8, device=dev()) for _ in range(2))
    table = i32(np.arange(pages, dtype=np.int32)[None])
    k = synth.normal(g, (1, Hkv, P + N, D), 1.0, True)
    v = synth.normal(g, (1, Hkv, P + N, D), 1.0, True)
    v[:, 0] = 0.0
    v[:, 1, :P // 2] = 0.0
    for lo, hi in ((0, P), (P, P + N)):
        tv.append_kv_paged(to_dev(k[:, :, lo:hi], True), to_dev(v[:, :, lo:hi], True), kc, vc, table, i32([lo]), k_scale=ks,
                           v_scale=vs)
    q = synth.normal(g, (1, 8, N, D), 1.0, True)
    got = host(tv.paged_attention(to_dev(q, True), kc, vc, table, i32([P]), k_scale=ks, v_scale=vs)).astype(np.float64)
    assert (got[:, :4] == 0).all()
    _compare(got, q, *(x.view(torch.uint8).cpu().numpy() for x in (kc, ks, vc, vs)), table.cpu().numpy(), [P], [N], [P + N],
             [0], None, None, True)


def test_append_of_more_declared_rows_than_an_int_of_lanes():
    # 2^27 declared rows of 160 elements (16 lanes each), of which 100 are active: a view that repeats one row
    ps, D = 64, 160
    x = to_dev(synth.normal(synth.rng(7800), (2, 1, 1, 1, D), 1.0, True), True)

    def run(N):
        kc, vc = (torch.zeros(3, 1, ps, D, dtype=torch.uint8, device=dev()).view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.zeros(3, 1, 1, dtype=torch.uint8, device=dev()) for _ in range(2))
        st = _status()
        tv.append_kv_paged(x[0].expand(1, 1, N, D), x[1].expand(1, 1, N, D), kc, vc, i32([[2, 0, 1]]), i32([7]),
                           n_rows=i32([100]), k_scale=ks, v_scale=vs, dev_status=st)
        assert int(st.item()) == 0
        return [t.view(torch.uint8) for t in (kc, vc, ks, vs)]
    ref, got = run(100), run(1 << 27)
    assert all((ref[i][2, 0, 7:] != 0).any(-1).all() and (ref[i][0, 0, :43] != 0).any(-1).all() for i in (0, 1))
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("q8_pages", [True, False])
@pytest.mark.parametrize("N,D", [(1, 128), (4, 128), (1, 64), (2, 256)])
def test_long_batches_repeat_bit_for_bit(N, D, q8_pages):
    # a persistent grid that streams a gigabyte: slots of its ring are refilled while their readers still run
    g = torch.Generator(device=dev()).manual_seed(7900 + N + D)
    B, Hkv, ps = 24 if q8_pages else 12, 8, 16
    width = 16384 // ps
    lens = torch.randint(8192, 16384 - N, (B,), generator=g, device=dev()).int()
    table = torch.randperm(B * width, generator=g, device=dev()).int().view(B, width)
    shape = (B * width, Hkv, ps, D)
    kw = {}
    if q8_pages:
        kc, vc = (torch.randint(0, 112, shape, generator=g, device=dev(), dtype=torch.uint8) for _ in range(2))
        kc, vc = (x.bitwise_or_(torch.randint(0, 2, shape, generator=g, device=dev(), dtype=torch.uint8) << 7)
                  .view(torch.float8_e4m3fn) for x in (kc, vc))
        kw = dict(k_scale=torch.randint(119, 121, (B * width, Hkv, 1), generator=g, device=dev(), dtype=torch.uint8),
                  v_scale=torch.randint(119, 121, (B * width, Hkv, 1), generator=g, device=dev(), dtype=torch.uint8))
    else:
        kc, vc = (torch.randn(shape, generator=g, device=dev(), dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn((B, 4 * Hkv, N, D), generator=g, device=dev(), dtype=torch.bfloat16)
    ws = torch.zeros(tv.paged_attention_workspace_size(B, 4 * Hkv, Hkv, D, N, ps, width, torch.bfloat16, cache_dtype=kc.dtype),
                     dtype=torch.uint8, device=dev())
    first = tv.paged_attention(q, kc, vc, table, lens, workspace=ws, **kw)
    assert torch.isfinite(first).all()
    different = sum(not torch.equal(tv.paged_attention(q, kc, vc, table, lens, workspace=ws, **kw), first) for _ in range(60))
    assert different == 0
