"""GPU parity of the round over an 8-bit paged cache against the oracle (64 bits): norms with the
rotation, the quantising append, the read back, attention over the codes, the commit, and a round.

Tolerances, per output element, u = eps / 2 of the type (2^-8 bf16, 2^-24 fp32):
  norm    the square sum of D terms in fp32 is off by D 2^-24 of itself at most, its root by half of
          that, with the mean, the square root, the reciprocal and two products 6 roundings more:
          a factor off by (D / 2 + 6) 2^-24; the rotation as in test_gpu_paged.py; u |out|
  append  the row before it is coded may be off by that d; a code is right where the numbers
          within d of the exact one round to it, so it is at most half a step and d off; the
          scale likewise.  Values are coded as they are: bit for bit
  attend  as in test_gpu_paged.py, the cached numbers being the oracle's exactly.  bf16 queries
          over codes may besides be off by 2^-17 of their row's largest element each: scale
          2^-17 max|q| sum_d |k_jd| on a score
"""
import math

import numpy as np
import pytest

import synth
import synth.workloads as W
from oracle import paged, paged_q8 as q8, rotary, tree

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import tree_speculative_decoding_masked_gb300 as tv  # noqa: E402
from gpu_util import dev, host, i32, to_dev  # noqa: E402
from test_gpu_paged import CHUNK, MANY, PERSISTENT, TOKEN, _pages, _rot_tol, _status, _unit  # noqa: E402


def _codes(c):
    return torch.from_numpy(c.copy()).to(dev()).view(torch.float8_e4m3fn)


def _bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def _pages8(g, B, Hkv, D, ps, blk, lens, total, low=None, std=1.0, wide=False):
    """Codes, scales and a table, as _pages: rows that no call needs hold codes of no number, and blocks of
    such rows any scale byte."""
    kc, vc, table = _pages(g, B, Hkv, D, ps, lens, total, False, low, std)
    out = []
    for x in (kc, vc):
        if wide:  # blocks of very different scales
            x = x * 2.0 ** np.repeat(g.integers(-9, 4, (x.shape[0], Hkv, ps // blk, 1)), blk, 2)
        codes, scale = q8.quantise(x, blk)
        none = np.isnan(x).all(-1).reshape(x.shape[0], Hkv, ps // blk, blk).all(-1)
        scale[none] = g.choice(np.array([0, 1, 127, 254, 255], np.uint8), int(none.sum()))
        out += [codes, scale]
    return (*out, table)


def _q8_attend_check(g, B, Hq, Hkv, D, ps, prefix, N, *, blk=None, parent=None, n_rows=None, softcap=0.0, window=0,
                     bf16=True, scale=None, std=1.0, workspace=None, wide=False):
    blk = min(ps, 16) if blk is None else blk
    act = [paged.active_rows(N, None if n_rows is None else n_rows[b], None if parent is None else parent[b])
           for b in range(B)]
    lens = [p + n if n else 0 for p, n in zip(prefix, act)]
    low = [p - window + 1 if window else 0 for p in prefix]
    kc, ks, vc, vs, table = _pages8(g, B, Hkv, D, ps, blk, lens, max(p + N for p in prefix), low, std, wide)
    q = synth.normal(g, (B, Hq, N, D), std, bf16)
    out = torch.full((B, Hq, N, D), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
    st = _status()
    got = tv.paged_attention(to_dev(q, bf16), _codes(kc), _codes(vc), i32(table), i32(prefix),
                             parent=None if parent is None else i32(parent),
                             n_rows=None if n_rows is None else i32(n_rows), scale=0.0 if scale is None else scale,
                             softcap=softcap, window=window, out=out, workspace=workspace, dev_status=st,
                             k_scale=torch.from_numpy(ks).to(dev()), v_scale=torch.from_numpy(vs).to(dev()))
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    got = host(got).astype(np.float64)
    with np.errstate(all="ignore"):
        k, v = q8.numbers(kc, ks), q8.numbers(vc, vs)
        ref, mass, big = paged.attention(q, k, v, table, prefix, parent, n_rows, scale, softcap, window)
    for b in range(B):
        assert np.all(got[b, :, act[b]:] == 7.0), "inactive rows were written"
        n = act[b]
        if n == 0:
            continue
        L = lens[b]
        e = 2 * D * 2.0 ** -23 * big[b, :, :n, None] + 2.0 ** -22 + L * 2.0 ** -23 + 2.0 ** -21 * softcap
        if bf16:
            rows = [(table[b, r // ps], r % ps) for r in range(max(low[b], 0), L)]
            norm = np.max([np.abs(k[p, :, r]).sum(-1) for p, r in rows], 0)  # [Hkv]
            e = e + (1 / math.sqrt(D) if scale is None else scale) * 2.0 ** -17 * (
                np.abs(q[b, :, :n]).max(-1) * np.repeat(norm, Hq // Hkv)[:, None])[..., None]
        tol = (2 * e + (2.0 ** -8 if bf16 else 0)) * mass[b, :, :n] + _unit(bf16) * np.abs(ref[b, :, :n])
        err = np.abs(got[b, :, :n] - ref[b, :, :n])
        assert np.isfinite(got[b, :, :n]).all()
        worst = np.max(err / np.maximum(tol, 1e-300))
        assert worst <= 1.0, (b, worst)
    return got


# ---- norms

ROT = [(128, 128), (128, 64), (64, 64), (64, 32), (96, 96), (256, 256), (128, 24), (80, 20), (7, 6), (32, 0),
       (1024, 1024), (512, 64)]


def _norm_tol(x, weight, eps, pos, rope, inter, bf16, ref):
    y = q8.norm(x, weight, eps)
    half = len(rope[0])
    pair = np.abs(y)
    if inter:
        s = pair[..., 0:2 * half:2] + pair[..., 1:2 * half:2]
        pair[..., 0:2 * half:2], pair[..., 1:2 * half:2] = s, s
    else:
        s = pair[..., :half] + pair[..., half:2 * half]
        pair[..., :half], pair[..., half:2 * half] = s, s
    return _rot_tol(y, pos, rope, inter, bf16, ref) + pair * rope[1] * (x.shape[-1] / 2 + 6) * 2.0 ** -24


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", ROT)
def test_norm_rotary(D, rot, inter, bf16):
    g = synth.rng(3000 + D + rot)
    B, H, N = 2, 5, 37
    x = synth.normal(g, (B, H, N, D), 1.0, bf16) * 2.0 ** g.integers(-6, 6, (B, H, N, 1)).astype(np.float32)
    weight = synth.normal(g, (D,), 1.0, bf16)
    pos = g.integers(0, 1 << 20, (B, N)).astype(np.int32)
    pos[:, 0], pos[-1, -1] = 0, (1 << 31) - 1
    rope = tv.rotary_frequencies(rot, 500000.0, scaling=("yarn", 16.0, 4096, 32.0, 1.0)) if rot else None
    ref_rope = rotary.frequencies(rot, 500000.0, ("yarn", 16.0, 4096, 32.0, 1.0)) if rot else (np.zeros(0), 1.0)
    ref = rotary.rotate(q8.norm(x, weight, 1e-5), pos[:, None], *ref_rope, inter)
    tol = _norm_tol(x, weight, 1e-5, pos, ref_rope, inter, bf16, ref)
    xd, wd = to_dev(x, bf16), to_dev(weight, bf16)
    got = tv.norm_rotary(xd, wd, i32(pos), rope, eps=1e-5, interleaved=inter)
    assert np.all(np.abs(host(got).astype(np.float64) - ref) <= tol)
    # rows of a projection, unaligned ones, a base, rows that count as padding, in place
    big = torch.zeros((B, N, H, D + 3), dtype=xd.dtype, device=dev())
    big[..., 3:] = xd.transpose(1, 2)
    out = torch.full_like(got, 7.0)
    tv.norm_rotary(big[..., 3:].transpose(1, 2), wd, i32(pos - 5), rope, eps=1e-5, interleaved=inter,
                   pos_base=i32(np.full(B, 5)), out=out)
    live = np.broadcast_to((pos - 5 >= 0)[:, None, :, None], ref.shape)
    out = host(out).astype(np.float64)
    assert np.all(np.abs(out - ref)[live] <= tol[live]) and np.all(out[~live] == 7.0)
    y = xd.clone()
    assert tv.norm_rotary(y, wd, i32(pos), rope, eps=1e-5, interleaved=inter, out=y) is y
    assert torch.equal(y, got)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_heads_share_a_group(inter, bf16):
    """Enough rows that heads share a thread, in numbers that its turns do not divide."""
    g = synth.rng(3050)
    B, H, N, D, rot = 3, 7, 20001, 64, 32
    x = synth.normal(g, (B, H, N, D), 1.0, bf16)
    weight = synth.normal(g, (D,), 1.0, bf16)
    pos = g.integers(0, 1 << 20, (B, N)).astype(np.int32)
    rope, ref_rope = tv.rotary_frequencies(rot, 500000.0), rotary.frequencies(rot, 500000.0)
    ref = rotary.rotate(q8.norm(x, weight, 1e-5), pos[:, None], *ref_rope, inter)
    tol = _norm_tol(x, weight, 1e-5, pos, ref_rope, inter, bf16, ref)
    xd, wd = to_dev(x, bf16), to_dev(weight, bf16)
    got = tv.norm_rotary(xd, wd, i32(pos), rope, eps=1e-5, interleaved=inter)
    assert np.all(np.abs(host(got).astype(np.float64) - ref) <= tol)
    assert torch.equal(tv.norm_rotary(xd, wd, i32(pos), rope, eps=1e-5, interleaved=inter, out=xd), got)


def test_norm_of_zeros_and_one_row():
    for bf16 in (True, False):
        x = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
        w = torch.ones_like(x[0, 0, 0])
        assert torch.equal(tv.norm_rotary(x, w, None, None), x)
        x[0, 0, 0, 3] = -2.0
        got = host(tv.norm_rotary(x, w, None, None, eps=0.0))
        assert got[0, 0, 0, 3] == -8.0 and np.count_nonzero(got) == 1


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("D,rot,N", [(128, 128, 1), (128, 64, 20), (96, 32, 7)])
def test_norm_append_into_plain_pages(D, rot, N, bf16):
    # the parts one by one give the same bits
    g = synth.rng(3100 + D + N)
    B, Hq, Hkv, ps, prefix = 2, 6, 2, 16, [30, 5]
    kc, vc, table = _pages(g, B, Hkv, D, ps, [p + N for p in prefix], 60, bf16)
    q, k, v = (to_dev(synth.normal(g, (B, h, N, D), 1.0, bf16), bf16) for h in (Hq, Hkv, Hkv))
    qw, kw = (to_dev(synth.normal(g, (D,), 1.0, bf16), bf16) for _ in "qk")
    rope = tv.rotary_frequencies(rot, 10000.0)
    kd, vd = to_dev(kc, bf16), to_dev(vc, bf16)
    out = tv.append_kv_paged(k, v, kd, vd, i32(table), i32(prefix), rope=rope, q=q, norm=(qw, kw, 1e-6))
    pos = i32(np.array([[p + t for t in range(N)] for p in prefix]))
    assert torch.equal(out, tv.norm_rotary(q, qw, pos, rope))
    turned = tv.norm_rotary(k, kw, pos, rope)
    k2, v2 = to_dev(kc, bf16), to_dev(vc, bf16)
    tv.append_kv_paged(turned, v, k2, v2, i32(table), i32(prefix))
    for a, b in ((kd, k2), (vd, v2)):
        assert torch.equal(torch.nan_to_num(a, 9.0), torch.nan_to_num(b, 9.0))


# ---- append

def _append_check(g, B, Hq, Hkv, N, D, rot, ps, blk, prefix, *, inter=False, norm=False, depth=None, n_rows=None,
                  with_q=True, bf16=True, std=1.0, unaligned=False, held_std=1.0, special=False):
    lens = [p + N for p in prefix]
    kc, ks, vc, vs, table = _pages8(g, B, Hkv, D, ps, blk, list(prefix), max(lens), std=held_std)
    # pages for the new rows
    count, width = kc.shape[0], table.shape[1]
    fresh = []
    for b in range(B):
        for p in range((prefix[b] + ps - 1) // ps, (lens[b] + ps - 1) // ps):
            table[b, p] = count + len(fresh)
            fresh.append(p)

    def more(x, fill):
        return np.concatenate((x, np.full((len(fresh), *x.shape[1:]), fill, x.dtype)))
    kc, vc, ks, vs = more(kc, 127), more(vc, 127), more(ks, 255), more(vs, 3)
    k, v, q = (synth.normal(g, (B, h, N, D), std, bf16) * 2.0 ** g.integers(-2, 3, (B, h, N, 1)).astype(np.float32)
               for h in (Hkv, Hkv, Hq))
    if special:
        k[..., 0, 1], v[..., 0, 2], v[..., 0, 3] = np.nan, np.inf, -np.inf
    qw, kw = (synth.normal(g, (D,), 1.0, bf16) for _ in "qk")
    active = np.zeros((B, N), bool)
    for b in range(B):
        active[b, :N if n_rows is None else n_rows[b]] = True
    if depth is not None:
        active &= depth >= 0
    rope = tv.rotary_frequencies(rot, 500000.0) if rot else None
    ref_rope = rotary.frequencies(rot, 500000.0) if rot else (np.zeros(0), 1.0)

    def put(x):
        t = to_dev(x, bf16)
        pad = 3 if unaligned else 8
        big = torch.zeros((B, N, x.shape[1], D + pad), dtype=t.dtype, device=dev())
        big[..., pad:] = t.transpose(1, 2)
        return big[..., pad:].transpose(1, 2)
    kd, vd, ksd, vsd = _codes(kc), _codes(vc), torch.from_numpy(ks.copy()).to(dev()), torch.from_numpy(vs.copy()).to(dev())
    st = _status()
    q_out = torch.full((B, Hq, N, D), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
    with_q = with_q and (norm or rope is not None)
    tv.append_kv_paged(put(k), put(v), kd, vd, i32(table), i32(prefix), depth=None if depth is None else i32(depth),
                       n_rows=None if n_rows is None else i32(n_rows), rope=rope, interleaved=inter,
                       q=put(q) if with_q else None, q_out=q_out if with_q else None,
                       norm=(to_dev(qw, bf16) if with_q else None, to_dev(kw, bf16), 1e-6) if norm else None,
                       k_scale=ksd, v_scale=vsd, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    off = np.arange(N)[None].repeat(B, 0) if depth is None else depth
    pos = np.asarray(prefix)[:, None] + np.maximum(off, 0)
    act4 = np.broadcast_to(active[:, None, :, None], q.shape)
    y = rotary.rotate(q8.norm(q, qw, 1e-6) if norm else q, pos[:, None], *ref_rope, inter)
    if with_q:
        got = host(q_out).astype(np.float64)
        tol = _norm_tol(q, qw, 1e-6, pos, ref_rope, inter, bf16, y) if norm else _rot_tol(q, pos, ref_rope, inter, bf16, y)
        assert np.all(np.abs(got - y)[act4] <= tol[act4]) and np.all(got[~act4] == 7.0)
    # values: bit for bit
    vc2, vs2 = q8.append(np.asarray(v, np.float64), vc, vs, table, prefix, active)
    assert np.array_equal(_bytes(vsd), vs2)
    assert np.array_equal(_bytes(vd) & 127, vc2 & 127) and np.array_equal(
        q8.decode(_bytes(vd)), q8.decode(vc2), equal_nan=True)
    # keys: the code of a number within d of the exact one
    turned = rotary.rotate(q8.norm(k, kw, 1e-6) if norm else np.asarray(k, np.float64), pos[:, None], *ref_rope, inter)
    d = (_norm_tol(k, kw, 1e-6, pos, ref_rope, inter, False, turned) if norm else
         _rot_tol(k, pos, ref_rope, inter, False, turned)) if rot or norm else np.zeros_like(turned)
    kc2, ks2 = q8.append(turned, kc, ks, table, prefix, active)
    got_c, got_s = _bytes(kd), _bytes(ksd)
    if not special:
        same = got_s == ks2
        assert np.mean(same) > 0.99 and np.all(np.abs(got_s[~same].astype(int) - ks2[~same]) == 1)
    else:
        assert np.array_equal(got_s, ks2)
    rows = got_c != kc2
    rows &= ~(np.isnan(q8.decode(got_c)) & np.isnan(q8.decode(kc2)))  # a NaN's sign is free
    # where codes differ the block's scale sits at a border, or the number between two codes
    got_n, ref_n = q8.numbers(got_c, got_s), q8.numbers(kc2, ks2)
    for b in range(B):
        for t in np.flatnonzero(active[b]):
            p, r = table[b, (prefix[b] + t) // ps], (prefix[b] + t) % ps
            diff = rows[p, :, r]
            if not diff.any():
                continue
            x, dd = turned[b, :, t], d[b, :, t]
            two = np.ldexp(1.0, got_s[p, :, r // blk].astype(int) - 127)[:, None]
            half = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(got_n[p, :, r]) / two, 2.0 ** -6))) - 4) * two, 0)
            assert np.all(np.abs(got_n[p, :, r] - x)[diff] <= (half + dd)[diff])
            rows[p, :, r] = False
    if not rows.any():
        return
    # held rows of a block whose scale sits at a border
    assert np.max(np.abs(got_n - ref_n)[rows] / np.abs(ref_n)[rows]) < 0.51


BLOCKS = [(16, 16), (16, 1), (8, 8), (64, 64), (128, 32), (1024, 64), (32, 2), (16, 4)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("ps,blk", BLOCKS)
@pytest.mark.parametrize("N", [1, 3, 37, 150])
def test_append_blocks(N, ps, blk, bf16):
    g = synth.rng(3200 + N + ps + blk)
    for D, rot, Hq, Hkv in ((128, 128, 8, 2), (64, 32, 3, 3)):
        _append_check(g, 3, Hq, Hkv, N, D, rot, ps, blk, [0, 2 * ps - 1, 69], bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot", [(32, 32), (64, 64), (96, 96), (128, 24), (160, 64), (192, 0), (224, 32), (256, 256)])
def test_append_heads(D, rot, norm, inter, bf16):
    g = synth.rng(3300 + D + rot)
    _append_check(g, 2, 4, 2, 70, D, rot, 32, 32, [5, 63], inter=inter, norm=norm, bf16=bf16)
    _append_check(g, 2, 4, 2, 2, D, rot, 16, 8, [5, 63], inter=inter, norm=norm, bf16=bf16, unaligned=True)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot,inter", [(256, 256, False), (160, 64, True)])
def test_append_wide_heads_and_long_blocks(D, rot, inter, norm, bf16):
    """More elements in a block of rows than a CTA has threads for: two rows a thread."""
    _append_check(synth.rng(3320 + D), 2, 3, 2, 150, D, rot, 128, 64, [5, 190], inter=inter, norm=norm, bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (96, 64, True)])
def test_append_heads_share_a_group(D, rot, inter, norm, bf16):
    """Enough rows that heads share a CTA, in numbers that its turns do not divide."""
    B, Hq, Hkv, N = 90, 7, 3, 100
    prefix = [int(p) for p in synth.rng(3330).integers(0, 70, B)]
    _append_check(synth.rng(3340 + D), B, Hq, Hkv, N, D, rot, 32, 16, prefix, inter=inter, norm=norm, bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("std", [2.0 ** -60, 2.0 ** -140, 2.0 ** 100])
def test_append_far_scales(std, bf16):
    if bf16 and std < 2.0 ** -120:
        std = 2.0 ** -105  # bf16's mantissa needs normal numbers
    _append_check(synth.rng(3400), 2, 2, 1, 20, 64, 0, 16, 16, [0, 16], std=std, bf16=bf16)


@pytest.mark.parametrize("held", [2.0 ** -12, 0.01, 1.0, 100.0])
@pytest.mark.parametrize("blk", [4, 64])
def test_append_behind_committed_rows(blk, held):
    # the scale grows over held rows, or keeps theirs
    g = synth.rng(3450 + blk)
    for N in (1, 5, 130):
        _append_check(g, 4, 4, 2, N, 128, 128, 64, blk, [3, 61, 66, 127], held_std=held, norm=True)


def test_append_trees_ragged_rows_and_specials():
    g = synth.rng(3500)
    N = 40
    par, _ = W.trees(g, 4, N, 6, 50)
    par[1, 25:], par[2, 1:] = -1, -1
    depth = np.stack([[len(tree.root_path(p, i)) - 1 if not tree.is_padding(p, i) else -1 for i in range(N)] for p in par])
    _append_check(g, 4, 8, 2, N, 128, 128, 16, 16, [17, 0, 31, 100], depth=depth)
    _append_check(g, 4, 8, 2, N, 64, 64, 16, 8, [17, 0, 31, 100], depth=depth, n_rows=[40, 0, 12, 7], bf16=False)
    # rows left out in the middle, the first of a block among them
    some = np.where(g.random((4, N)) < 0.5, np.arange(N), -1)
    _append_check(g, 4, 8, 2, N, 64, 64, 16, 8, [17, 0, 31, 100], depth=some)
    _append_check(g, 2, 2, 2, 20, 64, 0, 16, 16, [4, 0], special=True)


def test_append_reports_bad_pages_and_counts():
    g = synth.rng(3600)
    for what in ("page", "low", "long", "negative", "rows", "below"):
        kc, ks, vc, vs, table = _pages8(g, 2, 2, 64, 16, 16, [40, 40], 60)
        prefix, rows = [20, 20], [4, 4]
        if what == "page":
            table[0, 1] = kc.shape[0]
        elif what == "low":
            table[0, 1] = -1
        elif what == "long":
            prefix[0] = table.shape[1] * 16
        elif what == "negative":
            prefix[0] = -3
        elif what == "rows":
            rows[0] = 5
        else:
            rows[0] = -1
        k = to_dev(synth.normal(g, (2, 2, 4, 64), 1.0, True), True)
        kd, vd, ksd, vsd = _codes(kc), _codes(vc), torch.from_numpy(ks).to(dev()), torch.from_numpy(vs).to(dev())
        st = _status()
        tv.append_kv_paged(k, k, kd, vd, i32(table), i32(prefix), n_rows=i32(rows), k_scale=ksd, v_scale=vsd,
                           dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == tv.TV_DEV_BAD_PAGE, what
        # the other sequence's rows are there
        assert np.all(_bytes(vd)[table[1, 1], :, 4:8] & 127 != 127), what
        if what in ("page", "low", "negative", "rows", "below"):
            same = np.ones(kc.shape[0], bool)
            same[table[1, 1]] = False
            assert np.array_equal(_bytes(vd)[same], vc[same]), what


# ---- read back

@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,Hkv,D,ps,blk,lens", [
    (1, 1, 128, 16, 16, [1]), (3, 2, 64, 8, 1, [0, 5, 77]), (2, 3, 96, 64, 64, [130, 64]), (2, 1, 256, 1024, 32, [900, 40]),
    (2, 2, 32, 16, 8, [33, 16]), (1, 8, 160, 32, 16, [500]), (2, 2, 224, 16, 2, [31, 48])])
def test_read(B, Hkv, D, ps, blk, lens, bf16):
    g = synth.rng(3700 + D)
    kc, ks, vc, vs, table = _pages8(g, B, Hkv, D, ps, blk, lens, max(lens) + 1, wide=True)
    first = [n // 3 for n in lens]
    dt = torch.bfloat16 if bf16 else torch.float32
    rows = max(lens) + 3
    ko, vo = (torch.full((B, Hkv, rows, D), 7.0, dtype=dt, device=dev()) for _ in "kv")
    st = _status()
    args = (_codes(kc), _codes(vc), i32(table), i32(lens), torch.from_numpy(ks).to(dev()), torch.from_numpy(vs).to(dev()))
    for at in (None, first):
        ko.fill_(7.0)
        vo.fill_(7.0)
        assert tv.read_kv_paged(*args, first=None if at is None else i32(at), k_out=ko, v_out=vo, dev_status=st)[0] is ko
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        with np.errstate(all="ignore"):
            kn, vn = q8.numbers(kc, ks), q8.numbers(vc, vs)
        for b, n in enumerate(lens):
            f = 0 if at is None else at[b]
            for got, ref in ((host(ko), kn), (host(vo), vn)):
                want = paged.rows_of(ref, table[b], n)[:, f:]
                assert np.array_equal(got[b, :, :n - f].astype(np.float64), want)
                assert np.all(got[b, :, n - f:] == 7.0)
    k2, _ = tv.read_kv_paged(*args, rows=rows, dtype=dt)
    assert torch.equal(k2[0, :, :lens[0]], tv.read_kv_paged(*args, dtype=dt)[0][0, :, :lens[0]])


def test_every_code_and_scale_reads_exactly():
    codes = np.arange(256, dtype=np.uint8).reshape(1, 1, 8, 32).repeat(32, 0)
    scale = np.arange(256, dtype=np.uint8).reshape(32, 1, 8)
    table = np.arange(32)[None]
    s = torch.from_numpy(scale).to(dev())
    for dt in (torch.bfloat16, torch.float32):
        for order in (codes, np.roll(codes, 7, axis=2), np.roll(codes, 4, axis=2)):
            c = _codes(np.ascontiguousarray(order))
            got = host(tv.read_kv_paged(c, c, i32(table), i32([256]), s, s, dtype=dt)[0]).astype(np.float64)
            with np.errstate(all="ignore"):
                ref = paged.rows_of(q8.numbers(order, scale), table[0], 256)[None]
                # beyond the type's range, and rounded where its smallest steps are wider
                ref = torch.from_numpy(ref).to(torch.float32).to(dt).double().numpy()
            assert np.array_equal(got, ref, equal_nan=True)


def test_read_reports_bad_pages():
    g = synth.rng(3750)
    kc, ks, vc, vs, table = _pages8(g, 2, 2, 64, 16, 16, [40, 40], 41)
    table[0, 1] = kc.shape[0]
    s = [torch.from_numpy(x).to(dev()) for x in (ks, vs)]
    for first, length in ((None, [40, 40]), ([-1, 0], [40, 40]), (None, [-1, 40]), (None, [table.shape[1] * 16 + 1, 40])):
        st = _status()
        k, _ = tv.read_kv_paged(_codes(kc), _codes(vc), i32(table), i32(length), *s, rows=200, dev_status=st,
                                first=None if first is None else i32(first))
        torch.cuda.synchronize()
        assert int(st.item()) == tv.TV_DEV_BAD_PAGE
        with np.errstate(all="ignore"):
            assert np.array_equal(host(k)[1, :, :40], paged.rows_of(q8.numbers(kc, ks), table[1], 40))


# ---- attention

@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("blk", [1, 8, 64])
@pytest.mark.parametrize("shape", TOKEN + CHUNK)
def test_attend(shape, blk, bf16):
    B, Hq, Hkv, D, ps, prefix, N = shape
    _q8_attend_check(synth.rng(4000 + sum(shape[:5]) + N), B, Hq, Hkv, D, ps, prefix, N, blk=min(blk, ps), bf16=bf16,
                     wide=blk == 8)


@pytest.mark.parametrize("Hq,Hkv,N", [(2, 2, 1), (4, 2, 1), (3, 1, 1), (8, 2, 1), (2, 2, 2), (2, 2, 3), (4, 2, 2)])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 192, 256])
def test_attend_few_fp32_rows(D, Hq, Hkv, N):
    g = synth.rng(4150 + D + Hq + N)
    par, _ = W.trees(g, 3, N, 3, 50)
    _q8_attend_check(g, 3, Hq, Hkv, D, 16, [700, 0, 333], N, blk=16, bf16=False, wide=True)
    _q8_attend_check(g, 3, Hq, Hkv, D, 16, [700, 0, 333], N, blk=2, parent=par, softcap=20.0, bf16=False)
    _q8_attend_check(g, 3, Hq, Hkv, D, 16, [700, 0, 333], N, blk=16, window=65, bf16=False)


@pytest.mark.parametrize("N", [1, 2, 9])
def test_attend_fp32_queries_beyond_the_codes_range(N):
    # q of 2^121 and scales of 2^-117: a product with a code alone would not fit
    g = synth.rng(4160 + N)
    kc, ks, vc, vs, table = _pages8(g, 1, 2, 64, 16, 16, [50 + N], 50 + N, std=16.0)
    q = synth.normal(g, (1, 4, N, 64), 128.0, False)
    st = _status()
    got = [tv.paged_attention(to_dev(q * np.float32(2.0 ** e), False), _codes(kc), _codes(vc), i32(table), i32([50]),
                              k_scale=torch.from_numpy((ks - e).astype(np.uint8)).to(dev()),
                              v_scale=torch.from_numpy(vs).to(dev()), dev_status=st) for e in (0, 114)]
    assert torch.equal(got[0], got[1]) and torch.isfinite(got[0]).all() and int(st.item()) == 0


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", [(2, 8, 2, 128, 16, [100, 7], 3), (2, 8, 2, 128, 16, [300, 0], 40),
                                   (1, 4, 2, 64, 32, [70], 129), (1, 16, 2, 128, 64, [130], 70),
                                   (1, 4, 2, 96, 8, [33], 64), (1, 2, 2, 256, 16, [33], 50)])
def test_attend_trees(shape, bf16):
    B, Hq, Hkv, D, ps, prefix, N = shape
    g = synth.rng(4100 + sum(shape[:5]) + N)
    par, _ = W.trees(g, B, N, 6, 50)
    _q8_attend_check(g, B, Hq, Hkv, D, ps, prefix, N, parent=par, bf16=bf16)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("tree_", [False, True])
@pytest.mark.parametrize("shape", PERSISTENT)
def test_attend_persistent_schedule(shape, tree_, window):
    B, Hq, Hkv, D, ps, prefix, N = shape
    g = synth.rng(4170 + N + window)
    par, rows = None, [max(0, N - 3 * b) for b in range(B)]
    if tree_:
        par, _ = W.trees(g, B, N, 6, 50)
        rows = None
        for b in range(1, B):
            par[b, max(1, N - 2 * b):] = -1
    _q8_attend_check(g, B, Hq, Hkv, D, ps, prefix, N, blk=4 if window else None, parent=par, n_rows=rows, window=window,
                     softcap=20.0 if window else 0.0)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,Hq,Hkv,D,ps,N,P,tree_", MANY)
def test_attend_many_short_units(B, Hq, Hkv, D, ps, N, P, tree_, bf16):
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
    first = _q8_attend_check(synth.rng(24), B, Hq, Hkv, D, ps, prefix, N, parent=parent, n_rows=n_rows, window=window,
                             bf16=bf16)
    again = _q8_attend_check(synth.rng(24), B, Hq, Hkv, D, ps, prefix, N, parent=parent, n_rows=n_rows, window=window,
                             bf16=bf16)
    assert np.array_equal(first, again)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("window", [1, 16, 33, 5000])
@pytest.mark.parametrize("N", [1, 6, 80])
def test_attend_windows(bf16, window, N):
    g = synth.rng(4300 + N + window)
    _q8_attend_check(g, 2, 8, 2, 64, 16, [250, 31], N, window=window, bf16=bf16)
    par, _ = W.trees(g, 2, N, 7, 50)
    _q8_attend_check(g, 2, 8, 2, 64, 16, [250, 31], N, parent=par, window=window, bf16=bf16, blk=1)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("softcap", [0.5, 30.0, 1000.0])
@pytest.mark.parametrize("N", [1, 70])
def test_attend_softcap(bf16, softcap, N):
    g = synth.rng(4400 + N)
    if softcap <= 30.0:
        _q8_attend_check(g, 2, 8, 2, 128, 16, [200, 9], N, softcap=softcap, bf16=bf16, std=2.0, scale=0.5)
    _q8_attend_check(g, 2, 8, 2, 128, 16, [200, 9], N, softcap=softcap, window=40, bf16=bf16)


@pytest.mark.parametrize("N", [1, 9, 70])
def test_attend_ragged_rows(N):
    g = synth.rng(4200 + N)
    rows = [0, 1, N, max(1, N // 2)]
    par, _ = W.trees(g, 4, N, 5, 50)
    for b, n in enumerate(rows):
        par[b, max(1, n):] = -1
    for bf16 in (True, False):
        _q8_attend_check(g, 4, 8, 2, 128, 16, [50, 0, 17, 128], N, n_rows=rows, bf16=bf16)
        _q8_attend_check(g, 4, 8, 2, 128, 16, [50, 0, 17, 128], N, parent=par, bf16=bf16)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N", [1, 4, 40])
def test_attend_values_of_far_scales(N, bf16):
    # the keys that carry nearly all the weight have values 2^-18 of the others': what those add must stay
    g = synth.rng(4450 + N)
    B, Hq, Hkv, D, ps, P = 1, 4, 1, 128, 16, 600
    kc, ks, vc, vs, table = _pages8(g, B, Hkv, D, ps, 16, [P + N], P + N)
    k, v = q8.numbers(kc, ks), q8.numbers(vc, vs)
    u = np.sign(g.standard_normal(D))
    for r in range(P + N):
        p, h = table[0, r // ps], r // 16
        k[p, 0, r % ps] = u * (1.0 if h % 7 == 0 else -0.4) + 0.01 * k[p, 0, r % ps]
        if h % 7 == 0:
            v[p, 0, r % ps] *= 2.0 ** -18
    kc, ks = q8.quantise(k, 16)
    vc, vs = q8.quantise(v, 16)
    q = synth.round_to_bf16((u * np.abs(synth.normal(g, (B, Hq, N, D), 1.0, True)) * 0.9).astype(np.float32))
    got = host(tv.paged_attention(to_dev(q, bf16), _codes(kc), _codes(vc), i32(table), i32([P]),
                                  k_scale=torch.from_numpy(ks).to(dev()), v_scale=torch.from_numpy(vs).to(dev())))
    kn, vn = q8.numbers(kc, ks), q8.numbers(vc, vs)
    ref, mass, big = paged.attention(q, kn, vn, table, [P])
    e = 2 * D * 2.0 ** -23 * big[..., None] + 2.0 ** -22 + (P + N) * 2.0 ** -23
    if bf16:
        e = e + 2.0 ** -17 * big[..., None] * 4
    tol = (2 * e + (2.0 ** -8 if bf16 else 0)) * mass + _unit(bf16) * np.abs(ref)
    assert np.max(np.abs(got - ref) / tol) <= 1.0


@pytest.mark.parametrize("N", [1, 90])
@pytest.mark.parametrize("std", [2.0 ** -20, 2.0 ** 40])
def test_attend_queries_and_keys_of_far_scales(N, std):
    # queries and keys whose products are ordinary though neither is
    g = synth.rng(4460 + N)
    kc, ks, vc, vs, table = _pages8(g, 1, 2, 64, 16, 16, [300 + N], 300 + N)
    q = synth.normal(g, (1, 4, N, 64), 1.0, True)
    base = dict(v_scale=torch.from_numpy(vs).to(dev()))
    args = (_codes(kc), _codes(vc), i32(table), i32([300]))
    ref = tv.paged_attention(to_dev(q, True), *args, k_scale=torch.from_numpy(ks).to(dev()), **base)
    e = int(math.log2(std))
    got = tv.paged_attention(to_dev((q * std).astype(np.float32), True), *args, **base,
                             k_scale=torch.from_numpy(np.where(ks == 255, 255, ks.astype(int) - e).astype(np.uint8)).to(dev()))
    assert torch.equal(got, ref)


@pytest.mark.parametrize("N", [1, 70])
def test_attend_nan_query(N):
    g = synth.rng(4470)
    kc, ks, vc, vs, table = _pages8(g, 2, 2, 128, 16, 16, [200 + N, 50 + N], 200 + N)
    s = dict(k_scale=torch.from_numpy(ks).to(dev()), v_scale=torch.from_numpy(vs).to(dev()))
    q = to_dev(synth.normal(g, (2, 8, N, 128), 1.0, True), True)
    args = (_codes(kc), _codes(vc), i32(table), i32([200, 50]))
    ref = tv.paged_attention(q, *args, **s)
    q2 = q.clone()
    q2[1, 3, N - 1, 17] = float("nan")
    got = tv.paged_attention(q2, *args, **s)
    assert torch.isnan(got[1, 3, N - 1]).all()
    got[1, 3, N - 1] = ref[1, 3, N - 1]
    assert torch.equal(got, ref)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N", [1, 70])
def test_attend_bad_pages_are_reported(bf16, N):
    g = synth.rng(4500 + N)
    B, Hq, Hkv, D, ps, prefix = 3, 8, 2, 64, 16, [100, 60, 90]
    kc, ks, vc, vs, table = _pages8(g, B, Hkv, D, ps, 16, [p + N for p in prefix], 200)
    s = dict(k_scale=torch.from_numpy(ks).to(dev()), v_scale=torch.from_numpy(vs).to(dev()))
    q = to_dev(synth.normal(g, (B, Hq, N, D), 1.0, bf16), bf16)
    ref = host(tv.paged_attention(q, _codes(kc), _codes(vc), i32(table), i32(prefix), **s))
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
        got = host(tv.paged_attention(q, _codes(kc), _codes(vc), i32(t2), i32(p2), n_rows=i32(rows), dev_status=st, **s))
        assert int(st.item()) == tv.TV_DEV_BAD_PAGE, what
        assert np.array_equal(got[0], ref[0]) and np.array_equal(got[2], ref[2]), what


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N,Hkv,tree_", [(1, 2, False), (40, 2, True), (150, 2, False), (50, 40, True)])
def test_attend_repeats_are_bit_equal_and_replay(bf16, N, Hkv, tree_):
    g = synth.rng(4600 + N)
    B, Hq, D, ps, prefix = 2, 4 * Hkv, 128, 16, [700, 321]
    kc, ks, vc, vs, table = _pages8(g, B, Hkv, D, ps, 8, [p + N for p in prefix], 900)
    par = W.trees(g, B, N, 6, 50)[0] if tree_ else None
    q = to_dev(synth.normal(g, (B, Hq, N, D), 1.0, bf16), bf16)
    kd, vd, td, pd = _codes(kc), _codes(vc), i32(table), i32(prefix)
    s = dict(k_scale=torch.from_numpy(ks).to(dev()), v_scale=torch.from_numpy(vs).to(dev()).view(torch.uint8))
    pard = None if par is None else i32(par)
    n = tv.paged_attention_workspace_size(B, Hq, Hkv, D, N, ps, table.shape[1], q.dtype, cache_dtype=kd.dtype)
    ws = torch.zeros(max(256, n), dtype=torch.uint8, device=dev())
    st, out = _status(), torch.zeros_like(q)

    def call():
        return tv.paged_attention(q, kd, vd, td, pd, parent=pard, out=out, workspace=ws, dev_status=st, **s)
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
@pytest.mark.parametrize("N", [1, 4, 70])
def test_attend_pages_past_the_31st_bit(bf16, N):
    # a pool of 2^32 codes: the pages in use lie behind 2^31 bytes and at its very end
    g = synth.rng(4700)
    Hq, Hkv, D, ps, P = 8, 4, 128, 64, 400
    pages = (1 << 32) // (Hkv * ps * D)
    kd, vd = (torch.empty((pages, Hkv, ps, D), dtype=torch.float8_e4m3fn, device=dev()) for _ in "kv")
    ksd, vsd = (torch.empty((pages, Hkv, ps // 16), dtype=torch.uint8, device=dev()) for _ in "kv")
    kc, ks, vc, vs, table = _pages8(g, 1, Hkv, D, ps, 16, [P + N], P + N)
    at = np.concatenate(([pages - 1], np.arange(kc.shape[0] - 1) + pages // 2 + 3))
    for big, small in ((kd, _codes(kc)), (vd, _codes(vc)), (ksd, torch.from_numpy(ks).to(dev())), (vsd, torch.from_numpy(vs).to(dev()))):
        big[torch.from_numpy(at).to(dev())] = small
    far = table.copy()
    used = (P + N + ps - 1) // ps
    far[0, :used] = at[table[0, :used]]
    q = to_dev(synth.normal(g, (1, Hq, N, D), 1.0, bf16), bf16)
    near = tv.paged_attention(q, _codes(kc), _codes(vc), i32(table), i32([P]), k_scale=torch.from_numpy(ks).to(dev()),
                              v_scale=torch.from_numpy(vs).to(dev()))
    assert torch.equal(tv.paged_attention(q, kd, vd, i32(far), i32([P]), k_scale=ksd, v_scale=vsd), near)
    k = to_dev(synth.normal(g, (1, Hkv, N, D), 1.0, bf16), bf16)
    near_k, near_s = _codes(kc), torch.from_numpy(ks).to(dev())
    tv.append_kv_paged(k, k, near_k, _codes(vc), i32(table), i32([P]), k_scale=near_s, v_scale=torch.from_numpy(vs).to(dev()))
    tv.append_kv_paged(k, k, kd, vd, i32(far), i32([P]), k_scale=ksd, v_scale=vsd)
    a, _ = tv.read_kv_paged(kd, vd, i32(far), i32([P + N]), ksd, vsd, rows=P + N)
    b, _ = tv.read_kv_paged(near_k, near_k, i32(table), i32([P + N]), near_s, near_s, rows=P + N)
    assert torch.equal(a, b)


# ---- commit

@pytest.mark.parametrize("B,Hkv,D,ps,blk,prefix,N,lens", [
    (1, 2, 64, 16, 16, [20], 10, [3]),
    (3, 2, 128, 16, 1, [0, 15, 100], 40, [0, 16, 7]),
    (2, 3, 96, 8, 8, [63, 64], 200, [150, 199]),
    (2, 1, 256, 64, 64, [63, 5], 64, [63, 1]),
    (2, 2, 32, 128, 4, [127, 250], 1024, [900, 30]),
    (1, 8, 128, 1024, 64, [1000], 256, [16]),
    (4, 2, 224, 32, 32, [31, 30, 29, 0], 33, [1, 2, 3, 32]),
])
def test_commit(B, Hkv, D, ps, blk, prefix, N, lens):
    g = synth.rng(4800 + N)
    kc, ks, vc, vs, table = _pages8(g, B, Hkv, D, ps, blk, [p + N for p in prefix], max(prefix) + N, wide=True)
    acc = np.full((B, N), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        acc[b, :n] = np.sort(g.choice(np.arange(1, N), n, replace=False))
    kd, vd, ksd, vsd = _codes(kc), _codes(vc), torch.from_numpy(ks.copy()).to(dev()), torch.from_numpy(vs.copy()).to(dev())
    st = _status()
    new = tv.commit_accepted_kv_paged(kd, vd, i32(table), i32(prefix), i32(acc), i32(lens), k_scale=ksd, v_scale=vsd,
                                      dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and host(new).tolist() == [p + n + 1 for p, n in zip(prefix, lens)]
    for c, s, cd, sd in ((kc, ks, kd, ksd), (vc, vs, vd, vsd)):
        c2, s2 = q8.commit(c, s, table, prefix, acc, lens)
        assert np.array_equal(_bytes(sd), s2)
        assert np.array_equal(q8.decode(_bytes(cd)), q8.decode(c2), equal_nan=True)


def test_commit_reports_bad_paths_and_pages():
    g = synth.rng(4900)
    for path, n, prefix, bit in (([3, 2], 2, 20, tv.TV_DEV_BAD_TREE), ([3, 8], 2, 20, tv.TV_DEV_BAD_TREE),
                                 ([1, 2], 8, 20, tv.TV_DEV_BAD_TREE), ([1, 2], -1, 20, tv.TV_DEV_BAD_TREE),
                                 ([0, 2], 2, 20, tv.TV_DEV_BAD_TREE), ([2, 3], 2, -1, tv.TV_DEV_BAD_PAGE),
                                 ([2, 3], 2, 4000, tv.TV_DEV_BAD_PAGE)):
        kc, ks, vc, vs, table = _pages8(g, 1, 2, 64, 16, 16, [28], 28)
        acc = np.full((1, 8), -1, np.int32)
        acc[0, :2] = path
        st = _status()
        s = [torch.from_numpy(x).to(dev()) for x in (ks, vs)]
        tv.commit_accepted_kv_paged(_codes(kc), _codes(vc), i32(table), i32([prefix]), i32(acc), i32([n]), k_scale=s[0],
                                    v_scale=s[1], dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == bit, (path, n, prefix)


# ---- rounds

@pytest.mark.parametrize("blk", [1, 16, 64])
@pytest.mark.parametrize("graph", [False, True])
def test_rounds_over_8_bit_pages(blk, graph):
    """Prompt chunk, then rounds of a tree: append with norms, attend, verify, commit.  Every step's outputs
    against the oracle's from the cache as the step before left it."""
    g = synth.rng(5000 + blk)
    B, Hq, Hkv, D, ps, N, V, width = 2, 8, 2, 128, 64, 24, 512, 8
    table = g.permutation(B * width).reshape(B, width).astype(np.int32)
    kd, vd = (_codes(np.full((B * width, Hkv, ps, D), 127, np.uint8)) for _ in "kv")
    ksd, vsd = (torch.full((B * width, Hkv, ps // blk), 255, dtype=torch.uint8, device=dev()) for _ in "kv")
    qw, kw = (to_dev(synth.round_to_bf16(1 + synth.normal(g, (D,), 0.2)), True) for _ in "qk")
    rope = tv.rotary_frequencies(D, 10000.0)
    scales = dict(k_scale=ksd, v_scale=vsd)
    t, st = i32(table), _status()
    prompt = [150, 37]
    k, v = (to_dev(synth.normal(g, (B, Hkv, 150, D), 1.0, True), True) for _ in "kv")
    tv.append_kv_paged(k, v, kd, vd, t, i32([0, 0]), n_rows=i32(prompt), rope=rope, norm=(None, kw, 1e-6), **scales,
                       dev_status=st)
    length = i32(prompt)
    qkv = torch.zeros((B, N, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device=dev())
    rows = qkv.transpose(1, 2)
    par, tok = i32(np.zeros((B, N))), i32(np.zeros((B, N)))
    logits = torch.zeros((B, N, V), dtype=torch.bfloat16, device=dev())
    n = tv.paged_attention_workspace_size(B, Hq, Hkv, D, N, ps, width, torch.bfloat16, cache_dtype=kd.dtype)
    ws = torch.zeros(max(n, 256), dtype=torch.uint8, device=dev())
    q_out = torch.zeros((B, Hq, N, D), dtype=torch.bfloat16, device=dev())
    out, new = torch.zeros_like(q_out), torch.zeros_like(length)
    vws = torch.zeros(tv.verify_workspace_size(B, N, V, logits.dtype, False), dtype=torch.uint8, device=dev())
    chain = i32(np.stack([synth.chain_parents(N)] * B))
    prep = tv.tree_prep(chain, 0, dev_status=st)
    res = tv.verify_greedy(logits, chain, tok, workspace=vws, dev_status=st)

    def step():
        tv.tree_prep(par, 0, out=prep, dev_status=st)
        tv.append_kv_paged(rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], kd, vd, t, length, depth=prep["depth"], rope=rope,
                           q=rows[:, :Hq], q_out=q_out, norm=(qw, kw, 1e-6), dev_status=st, **scales)
        tv.paged_attention(q_out, kd, vd, t, length, parent=par, out=out, workspace=ws, dev_status=st, **scales)
        tv.verify_greedy(logits, par, tok, out=res, workspace=vws, dev_status=st)
        tv.commit_accepted_kv_paged(kd, vd, t, length, res["accepted_nodes"], res["accept_len"], new_len=new,
                                    dev_status=st, **scales)
    captured = None
    for turn in range(4):
        P = host(length).tolist()
        parent, tokens = W.trees(g, B, N, 5, V)
        qkv.copy_(to_dev(synth.normal(g, tuple(qkv.shape), 1.0 + turn, True), True))
        par.copy_(i32(parent))
        tok.copy_(i32(tokens))
        logits.copy_(to_dev(W.planted_logits(g, parent, tokens, V, True, prob=0.9), True))
        kc, ks, vc, vs = _bytes(kd), _bytes(ksd), _bytes(vd), _bytes(vsd)
        if graph and captured is None:
            saved = [y.clone() for y in (kd.view(torch.uint8), vd.view(torch.uint8), ksd, vsd)]
            step()  # warm up, then take it back
            for y, z in zip((kd.view(torch.uint8), vd.view(torch.uint8), ksd, vsd), saved):
                y.copy_(z)
            torch.cuda.synchronize()
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
        captured.replay() if graph else step()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        # values, and where the tree's codes were, through the oracle
        active = np.ones((B, N), bool)
        v_rows = host(rows[:, Hq + Hkv:]).astype(np.float64)
        vc2, vs2 = q8.append(v_rows, vc, vs, table, P, active)
        L = host(res["accept_len"]).tolist()
        acc = host(res["accepted_nodes"])
        vc3, vs3 = q8.commit(vc2, vs2, table, P, acc, L)
        assert np.array_equal(_bytes(vsd), vs3) and np.array_equal(q8.decode(_bytes(vd)), q8.decode(vc3), equal_nan=True)
        # attention: over the cache as the append left it; keys through the same call on a copy
        k2, v2, ks2, vs2d = _codes(kc), _codes(vc), torch.from_numpy(ks).to(dev()), torch.from_numpy(vs).to(dev())
        tv.append_kv_paged(rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], k2, v2, t, i32(P), depth=prep["depth"], rope=rope,
                           norm=(None, kw, 1e-6), k_scale=ks2, v_scale=vs2d)
        with np.errstate(all="ignore"):
            kn, vn = q8.numbers(_bytes(k2), _bytes(ks2)), q8.numbers(_bytes(v2), _bytes(vs2d))
            qn = host(q_out).astype(np.float64)
            ref, mass, big = paged.attention(qn, kn, vn, table, P, parent)
        e = (2 * D * 2.0 ** -23 + 2.0 ** -15) * big[..., None] + 2.0 ** -22 + (max(P) + N) * 2.0 ** -23
        tol = (2 * e + 2.0 ** -8) * mass + _unit(True) * np.abs(ref)
        assert np.max(np.abs(host(out) - ref) / tol) <= 1.0
        assert host(new).tolist() == [p + n + 1 for p, n in zip(P, L)]
        length.copy_(new)
