"""GPU tests of what the header promises for calls over pages beside their results."""
import ctypes

import numpy as np
import pytest

import paged_precision
import synth
from oracle import paged, rotary
from test_gpu_paged import _attend_check, _pages, _status, _unit

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import tree_speculative_decoding_masked_gb300 as tv  # noqa: E402
from gpu_util import dev, host, i32, to_dev  # noqa: E402


# ---- append: counts and padding

@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("count", [-1, 6, -(1 << 31), (1 << 31) - 1])
def test_append_reports_row_counts_out_of_range(count, bf16):
    # the count of sequence 1 is none: reported, and the other sequence's rows stand
    g = synth.rng(4000)
    N, rope = 5, tv.rotary_frequencies(64)
    x = to_dev(synth.normal(g, (2, 4, N, 64), 1.0, bf16), bf16)
    for depth in (None, i32([[0, 1, 1, 2, -1], [-1] * N])):
        for q in (None, x):
            pool = torch.zeros((4, 4, 8, 64), dtype=x.dtype, device=dev())
            pool_v, st = torch.zeros_like(pool), _status()
            tv.append_kv_paged(x, x, pool, pool_v, i32([[0, 3], [1, 2]]), i32([6, 6]), depth=depth,
                               n_rows=i32([4, count]), rope=rope, q=q, dev_status=st)
            torch.cuda.synchronize()
            assert int(st.item()) == tv.TV_DEV_BAD_PAGE
            assert torch.equal(pool_v[0, :, 6:], x[0, :, :2]) and torch.equal(pool_v[3, :, :2], x[0, :, 2:4])
            assert not pool_v[3, :, 2:].any() and not pool_v[0, :, :6].any()


def test_append_reports_a_negative_length_without_rows():
    x = torch.ones((2, 2, 3, 64), dtype=torch.bfloat16, device=dev())
    pool = torch.zeros((4, 2, 8, 64), dtype=torch.bfloat16, device=dev())
    for prefix, want in (([5, 0], 0), ([5, -1], tv.TV_DEV_BAD_PAGE)):
        st = _status()
        tv.append_kv_paged(x, x, pool, torch.zeros_like(pool), i32([[0, 3], [1, 2]]), i32(prefix), n_rows=i32([0, 0]),
                           dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == want and not pool.any()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("D", [64, 40])
@pytest.mark.parametrize("N,pad", [(5, 2), (70, 1), (70, 33), (70, 69), (300, 130)])
def test_append_goes_by_each_rows_depth(N, pad, D, bf16):
    # sequence 0 has no padding, 1 a row of negative depth among others, 2 what tree_prep makes of a
    # padded tree: -1 from the first padding row on
    g = synth.rng(4100 + N + pad)
    B, ps = 3, 8
    prefix = [3, 16, 9]
    dep = np.stack([np.minimum(np.arange(N), 7)] * B).astype(np.int32)
    dep[1, pad] = -5
    par = synth.chain_parents(N)[None].astype(np.int32)
    par[0, pad:] = -1
    dep[2] = host(tv.tree_prep(i32(par), 0)["depth"])[0]
    assert np.array_equal(dep[2] < 0, np.arange(N) >= pad)
    width = (max(prefix) + N + ps - 1) // ps
    table = g.permutation(B * width).reshape(B, width).astype(np.int32)
    k, v = (synth.normal(g, (B, 2, N, D), 1.0, bf16) for _ in range(2))
    q = synth.normal(g, (B, 4, N, D), 1.0, bf16)
    rope, (f, amp) = tv.rotary_frequencies(20), rotary.frequencies(20)
    kd = torch.full((B * width, 2, ps, D), 1024.0, dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
    vd, st, qo = kd.clone(), _status(), torch.full(q.shape, 1024.0, dtype=kd.dtype, device=dev())
    tv.append_kv_paged(to_dev(k, bf16), to_dev(v, bf16), kd, vd, i32(table), i32(prefix), depth=i32(dep), rope=rope,
                       q=to_dev(q, bf16), q_out=qo, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    fresh = np.full(kd.shape, 1024.0)
    kr, vr = paged.append(k, v, fresh, fresh, table, prefix, dep, None, f, amp)
    assert np.array_equal(host(vd), vr)
    kg, qg = host(kd).astype(np.float64), host(qo).astype(np.float64)
    bound = amp * 2.0 ** -21 * 2 * np.max(np.abs(k)) + _unit(bf16) * np.abs(kr)
    assert np.array_equal(kg == 1024.0, kr == 1024.0) and np.all(np.abs(kg - kr) <= bound)
    off = np.broadcast_to((dep < 0)[:, None, :, None], qg.shape)
    assert np.all(qg[off] == 1024.0) and not np.any(qg[~off] == 1024.0)


# ---- caps of any size

def _capped(g, B, Hq, Hkv, D, ps, prefix, N, softcap, std, bf16):
    """Largest error over tolerance.  A row's scores are at most Z = max_j scale |q| . |k_j|, and the cap makes
    them no larger: its error is relative, 2^-21 of min(softcap, Z), however large the cap.  The rest as in
    test_gpu_paged.py."""
    kc, vc, table = _pages(g, B, Hkv, D, ps, [p + N for p in prefix], max(prefix) + N, bf16, None, std)
    q = synth.normal(g, (B, Hq, N, D), std, bf16)
    st = _status()
    out = tv.paged_attention(to_dev(q, bf16), to_dev(kc, bf16), to_dev(vc, bf16), i32(table), i32(prefix),
                             softcap=softcap, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref, mass, big = paged.attention(q, kc, vc, table, prefix, softcap=softcap)
    keys = np.array(prefix)[:, None, None, None] + N
    e = (2 * D * 2.0 ** -23 + 2.0 ** -21) * big[..., None] + 2.0 ** -22 + keys * 2.0 ** -23
    tol = (2 * e + (2.0 ** -8 if bf16 else 0)) * mass + _unit(bf16) * np.abs(ref)
    return np.max(np.abs(host(out) - ref) / tol)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("softcap", [300.0, 1e4, 1e6, 1e8, 1e30, 3.2e38])
@pytest.mark.parametrize("Hq,Hkv,D,N", [(8, 2, 128, 1), (8, 2, 64, 70), (2, 1, 256, 20), (32, 1, 96, 3)])
def test_large_caps_cost_no_precision(Hq, Hkv, D, N, softcap, bf16):
    g = synth.rng(4200 + D + N)
    for std in (1.0, 2.5):
        assert _capped(g, 2, Hq, Hkv, D, 16, [50, 133], N, softcap, std, bf16) <= 1.0


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("softcap,std", [(300.0, 8.0), (300.0, 16.0), (1000.0, 16.0), (1e4, 40.0)])
@pytest.mark.parametrize("Hq,Hkv,D,N", [(8, 2, 128, 1), (8, 2, 64, 70), (2, 1, 256, 20), (8, 2, 128, 130)])
def test_scores_that_a_large_cap_bends(Hq, Hkv, D, N, softcap, std, bf16):
    # some scores below 0.45 of the cap, some past it
    g = synth.rng(4230 + D + N)
    assert _capped(g, 2, Hq, Hkv, D, 16, [50, 133], N, softcap, std, bf16) <= 1.0


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("softcap", [1e4, 1e8])
@pytest.mark.parametrize("N", [1, 11])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_caps_on_the_persistent_schedule(D, N, softcap, bf16):
    g = synth.rng(4250 + D + N)
    B = 170 if D <= 64 else 80
    assert _capped(g, B, 2, 1, D, 8, [(53 * b) % 150 for b in range(B)], N, softcap, 1.0, bf16) <= 1.0


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("softcap", [0.0, 20.0, 1e6])
@pytest.mark.parametrize("B,Hkv,N", [(2, 2, 1), (2, 2, 7), (2, 2, 70), (30, 8, 45)])
def test_a_nan_query_gives_a_nan_row_and_no_other(B, Hkv, N, softcap, bf16):
    g = synth.rng(4300 + N)
    Hq, D, ps = 2 * Hkv, 64, 16
    prefix = [(41 * b) % 200 + 1 for b in range(B)]
    kc, vc, table = _pages(g, B, Hkv, D, ps, [p + N for p in prefix], 201 + N, bf16)
    q = to_dev(synth.normal(g, (B, Hq, N, D), 1.0, bf16), bf16)
    args = (to_dev(kc, bf16), to_dev(vc, bf16), i32(table), i32(prefix))
    clean = tv.paged_attention(q, *args, softcap=softcap)
    assert bool(torch.isfinite(clean).all())
    sick = q.clone()
    where = torch.zeros((B, Hq, N), dtype=torch.bool, device=dev())
    for b, h, i in ((0, 1, N - 1), (1, 0, N // 2), (B - 1, Hq - 1, 0)):
        where[b, h, i] = True
        sick[b, h, i, (7 * i + h) % D] = float("nan")
    got = tv.paged_attention(sick, *args, softcap=softcap)
    assert bool(torch.isnan(got[where]).all())
    assert torch.equal(got[~where], clean[~where])


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("parent", [False, True])
@pytest.mark.parametrize("N", [1, 7, 60])
def test_no_active_rows_on_the_persistent_schedule(N, parent, bf16):
    # 320 units; then one row in the middle of them, and none again on the same workspace
    g = synth.rng(4400 + N)
    B, Hkv, D, ps = 40, 8, 64, 16
    par = np.stack([synth.chain_parents(N)] * B).astype(np.int32) if parent else None
    prefix = [(31 * b) % 100 for b in range(B)]
    rows = [0] * B
    ws = torch.zeros(tv.paged_attention_workspace_size(B, 2 * Hkv, Hkv, D, N, ps, 200 // ps + 2,
                                                       torch.bfloat16 if bf16 else torch.float32),
                     dtype=torch.uint8, device=dev())
    for n in (0, 1, 0):
        rows[17] = n
        _attend_check(g, B, 2 * Hkv, Hkv, D, ps, prefix, N, parent=par, n_rows=rows, bf16=bf16, workspace=ws)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,Hkv", [(3, 2), (45, 8)])
@pytest.mark.parametrize("N,act", [(4, 1), (4, 3), (12, 5), (90, 8), (90, 23), (90, 77)])
def test_padding_rows_need_no_pages(N, act, B, Hkv, bf16):
    # every table ends with a sequence's last active row or the page that holds it
    g = synth.rng(4500 + N + act)
    D, ps, width = 64, 8, 24
    prefix = [width * ps - act - (b % 3) for b in range(B)]
    par = np.stack([synth.random_parents(synth.rng(b), N, 8) for b in range(B)]).astype(np.int32)
    par[:, act:] = -1
    count = B * width
    table = g.permutation(count).reshape(B, width).astype(np.int32)
    kc, vc = (synth.normal(g, (count, Hkv, ps, D), 1.0, bf16) for _ in range(2))
    q = synth.normal(g, (B, 2 * Hkv, N, D), 1.0, bf16)
    args = [to_dev(x, bf16) for x in (q, kc, vc)]
    out, st = torch.full_like(args[0], 7.0), _status()
    tv.paged_attention(*args, i32(table), i32(prefix), parent=i32(par), out=out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    got = host(out)
    assert np.all(got[:, :, act:] == 7.0)
    some = [0, 1, B - 1]  # the oracle's loops are slow
    ref, mass, big = paged.attention(q[some], kc, vc, table[some], [prefix[b] for b in some], par[some])
    e = 2 * D * 2.0 ** -23 * big[..., None] + 2.0 ** -22 + width * ps * 2.0 ** -23
    tol = (2 * e + (2.0 ** -8 if bf16 else 0)) * mass + _unit(bf16) * np.abs(ref)
    assert np.all(np.abs(got[some] - ref)[:, :, :act] <= tol[:, :, :act])
    # an active row that does not fit
    st = _status()
    prefix[1] = width * ps - act + 1
    tv.paged_attention(*args, i32(table), i32(prefix), parent=i32(par), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == tv.TV_DEV_BAD_PAGE


# ---- outputs over inputs

def test_commit_refuses_new_len_over_its_inputs():
    kc = torch.zeros((4, 2, 8, 64), dtype=torch.bfloat16, device=dev())
    words = i32([5, 9, 1, 0, 0, 0, 7])  # lengths, accepted counts, one more
    pre, n, st = words[0:2], words[2:4], _status()
    table, acc = i32([[0, 1], [2, 3]]), i32([[2, -1, -1, -1], [-1, -1, -1, -1]])
    for new in (pre, n, words[1:3], words[3:5], acc[1, :2], acc[0, 2:], table[0]):
        with pytest.raises(tv.TreeVerifyError, match="TV_ERR_VALUE"):
            tv.commit_accepted_kv_paged(kc, kc.clone(), table, pre, acc, n, new_len=new, dev_status=st)
    got = tv.commit_accepted_kv_paged(kc, kc.clone(), table, pre, acc, n, new_len=words[4:6], dev_status=st)
    torch.cuda.synchronize()
    assert host(got).tolist() == [7, 10] and int(st.item()) == 0


def test_attention_refuses_an_output_over_its_queries():
    B, Hq, N, D = 2, 4, 3, 64
    count = B * Hq * N * D
    room = torch.zeros(2 * count, dtype=torch.bfloat16, device=dev())
    kc = torch.ones((4, 2, 8, D), dtype=torch.bfloat16, device=dev())
    args = (kc, kc.clone(), i32([[0, 1], [2, 3]]), i32([5, 9]))
    q = room[:count].view(B, Hq, N, D)
    for at in (0, 8, count - 8):
        with pytest.raises(tv.TreeVerifyError, match="TV_ERR_VALUE"):
            tv.paged_attention(q, *args, out=room[at:at + count].view(B, Hq, N, D))
    got = tv.paged_attention(q, *args, out=room[count:].view(B, Hq, N, D))  # side by side
    assert bool((got == 1.0).all()) and not room[:count].any()


# ---- a share of the device

def _grids(call, fit=False):
    """CTAs of each kernel that a call launches, asked of libcuda; with fit and how many an SM holds."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    cuda = ctypes.CDLL("libcuda.so.1")
    raw, count = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cuda.cuGraphGetNodes(raw, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert cuda.cuGraphGetNodes(raw, nodes, ctypes.byref(count)) == 0
    out = []
    for node in nodes:
        kind, params = ctypes.c_int(-1), (ctypes.c_uint32 * 64)()
        assert cuda.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value != 0:
            continue
        # a kernel: function, grid, block, shared memory, arguments, extra, kernel
        assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), params) == 0
        ctas = params[2] * params[3] * params[4]
        if fit:
            func = ctypes.c_void_p(params[0] | params[1] << 32)
            if not func.value:
                kern = ctypes.c_void_p(params[14] | params[15] << 32)
                assert cuda.cuKernelGetFunction(ctypes.byref(func), kern) == 0
            n = ctypes.c_int(0)
            assert cuda.cuOccupancyMaxActiveBlocksPerMultiprocessor(ctypes.byref(n), func, params[5] * params[6] * params[7],
                                                                    ctypes.c_size_t(params[8])) == 0
            out.append((ctas, n.value))
        else:
            out.append(ctas)
    return out


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,Hq,Hkv,D,N", [(1, 8, 2, 128, 1), (1, 32, 8, 64, 60), (4, 16, 8, 64, 1), (2, 16, 8, 128, 100),
                                          (1, 2, 1, 256, 90), (4, 32, 16, 96, 2), (1, 64, 8, 64, 5), (3, 40, 20, 32, 33)])
def test_few_units_keep_to_the_share(B, Hq, Hkv, D, N, bf16):
    # units that run as clusters on the whole device: fewer parts, or the persistent grid; one workspace for all
    g = synth.rng(4600 + D + N)
    dt = torch.bfloat16 if bf16 else torch.float32
    prefix = [700 - 111 * b for b in range(B)]
    ws = torch.zeros(tv.paged_attention_workspace_size(B, Hq, Hkv, D, N, 16, 60, dt) + 16, dtype=torch.uint8, device=dev())
    ws[-16:] = 77
    x = [torch.randn(s, device=dev()).to(dt) for s in ((B, Hq, N, D), (60, Hkv, 16, D), (60, Hkv, 16, D))]
    out, st, pre = torch.zeros_like(x[0]), _status(), i32(prefix)
    table = i32(np.stack([np.arange(60) for _ in range(B)]))
    try:
        for share in (0, 1, 7, 17, 40, 77, 120, 0):
            tv.set_sm_partition(0, share)
            _attend_check(g, B, Hq, Hkv, D, 16, prefix, N, bf16=bf16, workspace=ws[:-16])
            ctas = _grids(lambda: tv.paged_attention(*x, table, pre, out=out, workspace=ws[:-16], dev_status=st))
            assert len(ctas) == 1 and ctas[0] <= (share or 152) * (1 if bf16 else 2), (share, ctas)
            assert bool((ws[-16:] == 77).all())
    finally:
        tv.set_sm_partition(0, 0)


# ---- fp32 stays fp32

@pytest.mark.parametrize("case", paged_precision.CASES, ids=str)
def test_fp32_attention_is_off_by_fp32_roundings_only(case):
    data = paged_precision.inputs(case)
    q, kc, vc, table, par = data
    st = _status()
    got = tv.paged_attention(to_dev(q, False), to_dev(kc, False), to_dev(vc, False), i32(table), i32(case[5]),
                             parent=None if par is None else i32(par), softcap=case[8], window=case[9], dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert paged_precision.worst(case, data, host(got).astype(np.float64), paged_precision.reference(case, data)) <= 1.0


# ---- windows as wide as an int

@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 200])
@pytest.mark.parametrize("N,tree_", [(1, False), (6, True), (80, False), (80, True), (300, False)])
def test_a_window_of_any_size(N, tree_, window, bf16):
    g = synth.rng(4700 + N)
    par = np.stack([synth.random_parents(synth.rng(b), N, 8) for b in range(2)]).astype(np.int32) if tree_ else None
    wide = _attend_check(g, 2, 8, 2, 128, 16, [260, 33], N, parent=par, bf16=bf16, window=window)
    g = synth.rng(4700 + N)
    assert np.array_equal(wide, _attend_check(g, 2, 8, 2, 128, 16, [260, 33], N, parent=par, bf16=bf16))


# ---- idle sequences

@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("Hkv,N", [(2, 1), (2, 6), (2, 70), (60, 1), (60, 6), (60, 50)])
def test_a_sequence_without_rows_may_have_any_length(Hkv, N, bf16):
    # nothing of it is looked at; a negative length is reported all the same
    g = synth.rng(4800 + N)
    B, D, ps, prefix = 4, 64, 16, [30, 5, 77, 0]
    kc, vc, table = _pages(g, B, Hkv, D, ps, [p + N for p in prefix], 77 + N, bf16)
    q = to_dev(synth.normal(g, (B, 2 * Hkv, N, D), 1.0, bf16), bf16)
    args = (q, to_dev(kc, bf16), to_dev(vc, bf16), i32(table))
    rows = i32([N, 0, N, N])
    want = torch.full_like(q, 7.0)
    tv.paged_attention(*args, i32(prefix), n_rows=rows, out=want)
    for idle in (0, table.shape[1] * ps, table.shape[1] * ps + 1, 1 << 30, (1 << 31) - 1, -1):
        prefix[1] = idle
        st, got, pool = _status(), torch.full_like(q, 7.0), [args[1].clone(), args[2].clone()]
        tv.paged_attention(*args, i32(prefix), n_rows=rows, window=0, out=got, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == (tv.TV_DEV_BAD_PAGE if idle < 0 else 0), idle
        assert torch.equal(got, want)
        st = _status()
        k = q[:, ::2].clone()
        tv.append_kv_paged(k, k, *pool, i32(table), i32(prefix), n_rows=rows, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == (tv.TV_DEV_BAD_PAGE if idle < 0 else 0), idle


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,Hq,Hkv,D,N", [(40, 8, 8, 256, 1), (40, 32, 8, 256, 2), (40, 64, 8, 128, 1), (40, 64, 8, 128, 2),
                                          (40, 32, 8, 96, 4), (40, 16, 8, 64, 20), (40, 16, 8, 160, 20), (3, 16, 2, 256, 2)])
def test_a_share_holds_every_cta_at_once(B, Hq, Hkv, D, N, bf16):
    # by libcuda's count of the CTAs that fit on an SM
    dt = torch.bfloat16 if bf16 else torch.float32
    x = [torch.randn(s, device=dev()).to(dt) for s in ((B, Hq, N, D), (20, Hkv, 16, D), (20, Hkv, 16, D))]
    table, pre = i32(np.stack([np.arange(20) for _ in range(B)])), i32([300 - N - b for b in range(B)])
    out, st = torch.zeros_like(x[0]), _status()
    ws = torch.zeros(tv.paged_attention_workspace_size(B, Hq, Hkv, D, N, 16, 20, dt), dtype=torch.uint8, device=dev())
    try:
        for share in (9, 60):
            tv.set_sm_partition(0, share)
            for ctas, fit in _grids(lambda: tv.paged_attention(*x, table, pre, out=out, workspace=ws, dev_status=st), True):
                assert fit >= 1 and ctas <= share * fit, (share, ctas, fit)
    finally:
        tv.set_sm_partition(0, 0)
