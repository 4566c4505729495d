"""Timing cases of a verification round over a paged cache that is held in 8 bits: norms of
queries and keys with the rotation in the same pass, the append that quantises, the read back,
attention over the 8-bit pages, and the commit of an accepted path.

A cache element is an e4m3 code; a block of ``blk`` rows of a page shares, for each KV head, one
scale 2^(s - 127) held as the byte s, so a cached number is code * 2^(s - 127), exactly.

Each case runs either in a plain form (elementary torch operations in 32 bits, angles in 64) or,
with ``own`` true, through the framework's calls.  ``exact`` states every operator once more in 64
bits.

Shapes follow the repository's synthetic workloads (32 query and 8 KV heads of 128, trees of 16
to 1024 nodes, prefixes to 32768) and the single-token and prompt-chunk steps around a
verification round.  Caches hold pages in random order, as a server's free list leaves them, and
the sequences of a batch have different lengths.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0
LEAST = -117  # smallest scale exponent: the codes' smallest step stays a normal number
EPS = 1e-6


def listed():
    return [
        # the queries of one 64-node tree, normed and turned: latency
        dict(name="norm_tree", op="norm", B=1, H=32, N=64, D=128, rot=128, inter=False, P=120000, dtype="bf16"),
        # a prompt chunk's queries, interleaved pairs over half of the head: bandwidth
        dict(name="norm_chunk", op="norm", B=4, H=32, N=4096, D=128, rot=64, inter=True, P=8192, dtype="bf16"),
        # one token of a full decoding batch, its queries in the same call: latency
        dict(name="append_token", op="append", B=64, Hq=32, Hkv=8, N=1, D=128, ps=16, blk=16, P=2048, rot=128,
             inter=False, norm=True, tree=False, dtype="bf16"),
        # ragged prompt chunks with their queries: bandwidth
        dict(name="append_chunk", op="append", B=4, Hq=32, Hkv=8, N=2048, D=128, ps=32, blk=32, P=4001, rot=128,
             inter=False, norm=True, tree=False, dtype="bf16"),
        # one sequence's rows for a path that wants them in 16 bits: latency
        dict(name="read_one", op="read", B=1, Hkv=8, D=128, ps=16, blk=16, P=2048, dtype="bf16"),
        # a batch's rows, such as for moving sequences to another cache: bandwidth
        dict(name="read_batch", op="read", B=8, Hkv=8, D=128, ps=64, blk=64, P=16384, dtype="bf16"),
        # one sequence, one token: latency
        dict(name="attend_token", op="attend", B=1, Hq=32, Hkv=8, N=1, D=128, ps=16, blk=16, P=2048, tree=False,
             cap=0.0, window=0, dtype="bf16"),
        # a full decoding batch of ragged lengths: bandwidth
        dict(name="attend_batch", op="attend", B=64, Hq=32, Hkv=8, N=1, D=128, ps=16, blk=16, P=16384, tree=False,
             cap=0.0, window=0, dtype="bf16"),
        # the long-context workload's trees over 8-bit pages, lengths ragged
        dict(name="attend_tree_long", op="attend", B=8, Hq=32, Hkv=8, N=128, D=128, ps=64, blk=64, P=32768, tree=True,
             cap=0.0, window=0, dtype="bf16"),
        # capped scores and a sliding window, 32-bit queries, a scale a row, odd sizes
        dict(name="attend_cap_f32", op="attend", B=2, Hq=8, Hkv=4, N=100, D=64, ps=16, blk=1, P=3001, tree=True,
             cap=30.0, window=1024, dtype="f32"),
        # one sequence's accepted path
        dict(name="commit_tree", op="commit", B=1, Hkv=8, N=64, D=128, ps=16, blk=16, P=2048, L=5),
        # a full batch's accepted paths
        dict(name="commit_batch", op="commit", B=64, Hkv=8, N=256, D=128, ps=32, blk=32, P=4096, L=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "read", "attend", "attend", "attend", "commit"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([64, 128, 128])
    ps = rng.choice([8, 16, 32, 64, 128])
    blk = min(ps, rng.choice([1, 8, 16, 32, 64]))
    if op == "norm":
        N = _log(rng, 1, 4096)
        return dict(op=op, B=max(1, min(_log(rng, 1, 32), 16384 // N)), H=rng.choice([8, 16, 32]), N=N, D=D,
                    rot=rng.choice([D, D // 2, 32]), inter=rng.random() < 0.5, P=_log(rng, 1, 500000), dtype=dtype)
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    if op == "append":
        tree = rng.random() < 0.5
        N = _log(rng, 1, 256 if tree else 2048)
        return dict(op=op, B=max(1, min(_log(rng, 1, 64), 8192 // N)), Hq=Hq, Hkv=Hkv, N=N, D=D, ps=ps, blk=blk,
                    P=_log(rng, 1, 4000), rot=rng.choice([D, D // 2]), inter=rng.random() < 0.5,
                    norm=rng.random() < 0.5, tree=tree, dtype=dtype)
    if op == "read":
        P = _log(rng, 1, 16384)
        return dict(op=op, B=max(1, min(_log(rng, 1, 64), 8 * 16384 // P)), Hkv=Hkv, D=D, ps=ps, blk=blk, P=P,
                    dtype=dtype)
    if op == "commit":
        N = _log(rng, 16, 1024)
        return dict(op=op, B=_log(rng, 1, 64), Hkv=Hkv, N=N, D=D, ps=ps, blk=blk, P=_log(rng, 1, 4000),
                    L=rng.randint(0, min(16, N // 2 - 1)))
    kind = rng.choice(["token", "tree", "chunk"])
    N = 1 if kind == "token" else _log(rng, 2, 512) if kind == "tree" else _log(rng, 2, 2048)
    P = _log(rng, 1, 24000)
    # the score count (an eighth of it in 32 bits, which run on CUDA cores) and the cache of the largest listed cases
    # bound B
    most, cache = 8 * 32 * 128 * 32768 // (8 if dtype == "f32" else 1), 64 * 12288 * 8 * 128
    B = max(1, min(_log(rng, 1, 64), most // (Hq * N * (P + N)), cache // ((P + N) * Hkv * D)))
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, N=N, D=D, ps=ps, blk=blk, P=P, tree=kind == "tree",
                cap=rng.choice([0.0, 0.0, 30.0, 50.0]), window=rng.choice([0, 0, 0, 64, 1000, 4096]), dtype=dtype)


def _prefix(case):
    """Committed lengths of the batch's sequences: the longest first, down to half of it."""
    P, B = case["P"], case["B"]
    return [P - (b * 7919) % (P // 2 + 1) for b in range(B)]


def _rows(case):
    """New rows of each sequence: some of a batch's chunks and trees are shorter than N."""
    N, B = case["N"], case["B"]
    return [N - (b * 31) % (N // 3 + 1) for b in range(B)]


def _parents(case):
    """Draft trees [B][N]: node t hangs below one of the 24 nodes before it, at most 16 deep, trailing padding -1."""
    r = np.random.RandomState(case["N"] * 1000 + case["B"])
    out = np.full((case["B"], case["N"]), -1, dtype=np.int32)
    dep = np.full((case["B"], case["N"]), -1, dtype=np.int32)
    for b, n in enumerate(_rows(case)):
        dep[b, 0] = 0
        for t in range(1, n):
            p = r.randint(max(0, t - 24), t)
            while dep[b, p] >= 16:
                p = int(out[b, p])
            out[b, t] = p
            dep[b, t] = dep[b, p] + 1
    return out, dep


_BASE = 500000.0


def _inv_freq(rot):
    return _BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _randn(shape, gen, dtype):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // max(1, math.prod(shape[1:])))
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        out[i:i + n] = torch.randn((n, *shape[1:]), generator=gen, device="cuda", dtype=torch.float32)
    return out


def _ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, at least LEAST."""
    m, x = torch.frexp(amax)  # amax = m 2^x, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(amax > 0, x - 9 + (m > E4M3_MAX / 512), LEAST)
    return e.clamp(min=LEAST).int()


def _two(e):
    """2^e of integers -126..127, in 32 bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x, e):
    return (x * _two(-e)).to(torch.float8_e4m3fn)


def _decode(code, e):
    return code.float() * _two(e)


def _exp_of(scale):
    return scale.int() - 127


def _byte_of(e):
    return (e + 127).to(torch.uint8)


def _pages(shape, blk, gen, gain):
    """Codes and scale bytes of a cache of N(0, gain_d) rows."""
    pages, Hkv, ps, D = shape
    code = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((pages, Hkv, ps // blk), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (Hkv * ps * D))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.randn((n, Hkv, ps // blk, blk, D), generator=gen, device="cuda") * gain
        e = _exponent(x.abs().amax((-1, -2)))
        code[i:i + n] = _encode(x, e[..., None, None]).reshape(n, Hkv, ps, D)
        scale[i:i + n] = _byte_of(e)
    return code, scale


def _paged(case, gen):
    """A cache of just the pages that the batch needs and a few more, and the table of each sequence's pages."""
    B, ps, D = case["B"], case["ps"], case["D"]
    need = [(p + case.get("N", 0) + ps - 1) // ps for p in _prefix(case)]
    width, pages = max(need) + 1, sum(need) + 5
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    shape = (pages, case["Hkv"], ps, D)
    # keys have a few channels that are larger than the others
    gain = torch.ones(D, device="cuda")
    gain[::32] = 3.0
    k, ks = _pages(shape, case["blk"], gen, gain)
    v, vs = _pages(shape, case["blk"], gen, 1.0)
    return k, v, ks, vs, table


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, s = DTYPES[case.get("dtype", "bf16")], dict(case=case)
    B, D = case["B"], case["D"]
    if case["op"] in ("norm", "append"):
        s["inv_freq"] = _inv_freq(case["rot"]).cuda()
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt) for _ in "qk")
        if own:
            import tree_speculative_decoding_masked_gb300 as tv
            s["rope"] = tv.rotary_frequencies(case["rot"], _BASE, device="cuda")
    s["dev_status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "norm":
        H, N = case["H"], case["N"]
        # token-major rows, as a projection writes them
        s["x"] = _randn((B, N, H, D), gen, dt).transpose(1, 2)
        start = torch.randint(0, case["P"], (B, 1), generator=gen, device="cuda", dtype=torch.int32)
        s["pos"] = (start + torch.arange(N, device="cuda", dtype=torch.int32)).contiguous()
        s["out"] = torch.zeros((B, H, N, D), dtype=dt, device="cuda")
        return s
    Hkv = case["Hkv"]
    s["lens"] = _prefix(case)
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"] = _paged(case, gen)
    s["prefix_len"] = _ints(s["lens"])
    if case["op"] == "read":
        s["k_out"], s["v_out"] = (torch.zeros((B, Hkv, max(s["lens"]), D), dtype=dt, device="cuda") for _ in "kv")
        return s
    N = case["N"]
    s["rows"] = _rows(case)
    s["n_rows"] = _ints(s["rows"])
    if case["op"] == "commit":
        L = case["L"]
        # an accepted path's nodes, anywhere in the tree; some sequences accept fewer
        acc = np.full((B, N), -1, dtype=np.int32)
        r = np.random.RandomState(int(seed) % (1 << 31))
        s["accepted"] = [sorted(r.choice(np.arange(L + 1, N), L - b % (L // 2 + 1), replace=False)) for b in range(B)]
        for b, path in enumerate(s["accepted"]):
            acc[b, :len(path)] = path
        s["accepted_nodes"], s["accept_len"] = _ints(acc), _ints([len(p) for p in s["accepted"]])
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    Hq = case["Hq"]
    s["parent"] = s["depth"] = None
    if case["tree"]:
        par, dep = _parents(case)
        s["parent"], s["depth"] = _ints(par), _ints(dep)
    s["out"] = torch.zeros((B, Hq, N, D), dtype=dt, device="cuda")
    if case["op"] == "append":
        # q, k and v are parts of one projection's output
        qkv = _randn((B, N, Hq + 2 * Hkv, D), gen, dt).transpose(1, 2)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        return s
    s["q"] = _randn((B, Hq, N, D), gen, dt)
    if own:
        import tree_speculative_decoding_masked_gb300 as tv
        n = tv.paged_attention_workspace_size(B, Hq, Hkv, D, N, case["ps"], s["table"].shape[1], dt,
                                              cache_dtype=torch.float8_e4m3fn)
        s["workspace"] = torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")
    return s


# ---- plain forms


def _normed(x, weight):
    """x [..., D] over its root mean square, times the weight, in 32 bits."""
    y = x.float()
    return y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()


def _rotate(y, pos, s):
    """y [B][H][N][D] (32 bits) at positions pos [B][N] (float64 angles)."""
    case, rot = s["case"], s["case"]["rot"]
    ang = pos.double()[:, None, :, None] * s["inv_freq"]
    cos, sin = ang.cos().float(), ang.sin().float()
    y = y.clone()
    if case["inter"]:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_norm(s):
    s["out"].copy_(_rotate(_normed(s["x"], s["q_weight"]), s["pos"], s))
    return s["out"]


def _write(x, code, scale, b, t, page, row, s):
    """Rows x [M][Hkv][D] (32 bits) to (page, row); a block's scale covers what it held and what comes."""
    blk = s["case"]["blk"]
    Hkv, nb = scale.shape[1], scale.shape[2]
    h = torch.arange(Hkv, device="cuda")
    at = (page[:, None] * Hkv + h) * nb + (row // blk)[:, None]  # [M][Hkv]: the row's block
    amax = torch.full((scale.numel(),), -1.0, device="cuda")
    amax.scatter_reduce_(0, at.reshape(-1), x.abs().amax(-1).reshape(-1), "amax")
    touched = amax >= 0
    # blocks that begin with committed rows keep at least the scale of those
    P = s["prefix_len"].long()
    ps = s["case"]["ps"]
    r = (P // blk * blk)[:, None] + torch.arange(blk, device="cuda")
    ob, oj = torch.nonzero(r < P[:, None], as_tuple=True)
    r = r[ob, oj]
    opage, orow = s["table"].long()[ob, r // ps], r % ps
    oat = (opage[:, None] * Hkv + h) * nb + (orow // blk)[:, None]
    old = _exp_of(scale).reshape(-1)
    floor = torch.full_like(old, LEAST)
    floor[oat.reshape(-1)] = old[oat.reshape(-1)]
    new = torch.where(touched, torch.maximum(_exponent(amax.clamp(min=0)), floor), old)
    kept = _decode(code[opage, :, orow], old[oat][..., None])
    code[opage, :, orow] = _encode(kept, new[oat][..., None])
    code[page, :, row] = _encode(x, new[at][..., None])
    scale.copy_(torch.where(touched, _byte_of(new), scale.reshape(-1)).view_as(scale))


def _plain_append(s):
    case = s["case"]
    off = torch.arange(case["N"], device="cuda")[None] if s["depth"] is None else s["depth"]
    pos = s["prefix_len"][:, None] + off
    t = torch.arange(case["N"], device="cuda", dtype=torch.int64)
    b, t = torch.nonzero(t[None] < s["n_rows"][:, None], as_tuple=True)
    at = s["prefix_len"].long()[b] + t
    page, row = s["table"].long()[b, at // case["ps"]], at % case["ps"]
    q, k = (_normed(s["q"], s["q_weight"]), _normed(s["k"], s["k_weight"])) if case["norm"] else \
        (s["q"].float(), s["k"].float())
    _write(_rotate(k, pos, s)[b, :, t], s["k_cache"], s["k_scale"], b, t, page, row, s)
    _write(s["v"][b, :, t].float(), s["v_cache"], s["v_scale"], b, t, page, row, s)
    s["out"][b, :, t] = _rotate(q, pos, s)[b, :, t].to(s["out"].dtype)
    return _cache_of(s) | {"q": s["out"]}


def _cache_of(s):
    """The cache as it is: codes and scales, each as the numbers they stand for."""
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scale": s["k_scale"].view(torch.float8_e8m0fnu),
            "v_scale": s["v_scale"].view(torch.float8_e8m0fnu)}


def _gather(code, scale, table, blk):
    """Rows [n][Hkv][L][D] (32 bits) of the pages that table [n][pages] names."""
    n, pages = table.shape
    x = _decode(code[table].unflatten(3, (-1, blk)), _exp_of(scale[table])[..., None, None]).flatten(3, 4)
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_read(s):
    ps, blk = s["case"]["ps"], s["case"]["blk"]
    L = s["k_out"].shape[2]
    live = (torch.arange(L, device="cuda")[None] < s["prefix_len"][:, None])[:, None, :, None]
    table = s["table"][:, :(L + ps - 1) // ps].clamp(min=0).long()
    for code, scale, out in ((s["k_cache"], s["k_scale"], s["k_out"]), (s["v_cache"], s["v_scale"], s["v_out"])):
        out.copy_(torch.where(live, _gather(code, scale, table, blk)[:, :, :L], out.float()))
    return {"k": s["k_out"], "v": s["v_out"]}


def _ancestors(parent):
    """[B][N][N]: node j is node i or one of its ancestors."""
    B, N = parent.shape
    see = torch.zeros((B, N, N), dtype=torch.bool, device="cuda")
    cur, at = torch.arange(N, device="cuda").expand(B, N).clone(), parent.long()
    for _ in range(18):  # depth at most 16
        see.scatter_(2, cur.clamp(min=0)[..., None], True)
        cur = torch.where(cur > 0, at.gather(1, cur.clamp(min=0)), torch.zeros_like(cur))
    return see


def _plain_attend(s):
    case = s["case"]
    B, Hq, Hkv, N, D, ps = (case[k] for k in ("B", "Hq", "Hkv", "N", "D", "ps"))
    G, longest = Hq // Hkv, max(s["lens"]) + N
    t = torch.arange(N, device="cuda")
    step = max(1, (1 << 31) // (Hq * N * longest))
    for b0 in range(0, B, step):
        n = min(step, B - b0)
        pages = (max(s["lens"][b0:b0 + n]) + N + ps - 1) // ps
        j = torch.arange(pages * ps, device="cuda")
        L = j.numel()
        table = s["table"][b0:b0 + n, :pages].clamp(min=0).long()
        k = _gather(s["k_cache"], s["k_scale"], table, case["blk"])
        v = _gather(s["v_cache"], s["v_scale"], table, case["blk"])
        P, rows = s["prefix_len"][b0:b0 + n, None, None], s["n_rows"][b0:b0 + n, None, None]
        new = (j[None, None] - P).expand(n, N, L)  # the new row that key j is
        inside = (new < rows) & (j < L)
        if s["parent"] is None:
            dist = t[None, :, None] - new
            see = inside & (dist >= 0)
        else:
            tree = _ancestors(s["parent"][b0:b0 + n])
            see = inside & ((new < 0) | tree.gather(2, new.clamp(0, N - 1)))
            dep = s["depth"][b0:b0 + n].long()
            key = torch.where(new < 0, new, dep.gather(1, new[:, 0].clamp(0, N - 1))[:, None].expand(n, N, L))
            dist = dep[:, :, None] - key
        if case["window"]:
            see = see & (dist < case["window"])
        q = s["q"][b0:b0 + n].float().reshape(n, Hkv, G * N, D)
        z = q @ k.transpose(-1, -2) / math.sqrt(D)
        if case["cap"]:
            z = case["cap"] * torch.tanh(z / case["cap"])
        z = z.reshape(n, Hkv, G, N, L).masked_fill(~see[:, None, None], float("-inf"))
        e = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e30))
        v = v.masked_fill(~inside[:, :1, :].transpose(1, 2)[:, None], 0.0)
        o = (e.reshape(n, Hkv, G * N, L) @ v).reshape(n, Hkv, G, N, D) / e.sum(-1, keepdim=True)
        live = (t[None] < s["n_rows"][b0:b0 + n, None])[:, None, :, None]
        s["out"][b0:b0 + n] = torch.where(live, o.reshape(n, Hq, N, D).to(s["out"].dtype), s["out"][b0:b0 + n])
    return s["out"]


def _plain_commit(s):
    """Path rows move to the places behind the root; a block that receives rows takes the largest scale of what it
    then holds, and its live rows are coded to that."""
    case, P = s["case"], s["prefix_len"].long()
    ps, blk, table = case["ps"], case["blk"], s["table"].long()
    k = torch.arange(case["N"], device="cuda")
    b, k = torch.nonzero(k[None] < s["accept_len"][:, None], as_tuple=True)
    src, dst = P[b] + s["accepted_nodes"].long()[b, k], P[b] + k + 1
    spage, srow, page, row = table[b, src // ps], src % ps, table[b, dst // ps], dst % ps
    # the rows before the first moved one that share its block stay live
    first = P + 1
    r = (first // blk * blk)[:, None] + torch.arange(blk, device="cuda")
    ob, oj = torch.nonzero((r < first[:, None]) & (s["accept_len"] > 0)[:, None], as_tuple=True)
    r = r[ob, oj]
    opage, orow = table[ob, r // ps], r % ps
    for code, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        Hkv, nb = scale.shape[1], scale.shape[2]
        h = torch.arange(Hkv, device="cuda")
        old = _exp_of(scale).reshape(-1)

        def block(p, x):
            return (p[:, None] * Hkv + h) * nb + (x // blk)[:, None]
        new = old.clone()
        new.scatter_reduce_(0, block(page, row).reshape(-1), old[block(spage, srow)].reshape(-1), "amax")
        moved = _decode(code[spage, :, srow], old[block(spage, srow)][..., None])
        kept = _decode(code[opage, :, orow], old[block(opage, orow)][..., None])
        code[opage, :, orow] = _encode(kept, new[block(opage, orow)][..., None])
        code[page, :, row] = _encode(moved, new[block(page, row)][..., None])
        scale.copy_(_byte_of(new).view_as(scale))
    s["new_len"].copy_(s["prefix_len"] + s["accept_len"] + 1)
    return _cache_of(s) | {"new_len": s["new_len"]}


def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "append": _plain_append, "read": _plain_read, "attend": _plain_attend,
                "commit": _plain_commit}[op](s)
    import tree_speculative_decoding_masked_gb300 as tv
    if op == "norm":
        return tv.norm_rotary(s["x"], s["q_weight"], s["pos"], s["rope"], eps=EPS, interleaved=case["inter"],
                              out=s["out"])
    if op == "append":
        norm = (s["q_weight"], s["k_weight"], EPS) if case["norm"] else None
        tv.append_kv_paged(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], depth=s["depth"],
                           n_rows=s["n_rows"], rope=s["rope"], interleaved=case["inter"], q=s["q"], q_out=s["out"],
                           norm=norm, k_scale=s["k_scale"], v_scale=s["v_scale"], dev_status=s["dev_status"])
        return _cache_of(s) | {"q": s["out"]}
    if op == "read":
        tv.read_kv_paged(s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], s["k_scale"], s["v_scale"],
                         k_out=s["k_out"], v_out=s["v_out"], dev_status=s["dev_status"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "commit":
        tv.commit_accepted_kv_paged(s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], s["accepted_nodes"],
                                    s["accept_len"], new_len=s["new_len"], k_scale=s["k_scale"],
                                    v_scale=s["v_scale"], dev_status=s["dev_status"])
        return _cache_of(s) | {"new_len": s["new_len"]}
    return tv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], parent=s["parent"],
                              n_rows=s["n_rows"], softcap=case["cap"], window=case["window"], k_scale=s["k_scale"],
                              v_scale=s["v_scale"], out=s["out"], workspace=s["workspace"],
                              dev_status=s["dev_status"])


# ---- 64-bit statement


def _two64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3_64(x):
    """The e4m3 number nearest to x (float64, |x| <= 448), ties to the even code."""
    step = _two64(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
    return torch.round(x / step) * step


def _block_64(rows, least):
    """(codes, exponents [Hkv]) of a block's rows [Hkv][n][D] (float64), the exponents at least `least`."""
    top = rows.abs().amax((-1, -2))
    e = torch.maximum(least, torch.where(top > 0, torch.frexp(top)[1] - 10, LEAST))
    while bool((top > E4M3_MAX * _two64(e)).any()):
        e = e + (top > E4M3_MAX * _two64(e))
    return _e4m3_64(rows * _two64(-e)[:, None, None]), e


def _turn64(x, pos, case):
    """One row set x [..., D] (float64) turned by complex products; pos broadcasts over the leading axes."""
    rot = case["rot"]
    ang = pos[..., None] * _inv_freq(rot).to(x.device)
    w = torch.polar(torch.ones_like(ang), ang)
    head = x[..., :rot]
    pair = head.unflatten(-1, (rot // 2, 2)) if case["inter"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    y = torch.view_as_real(torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * w)
    y = y.flatten(-2) if case["inter"] else y.transpose(-1, -2).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _norm64(x, weight):
    x = x.double()
    return x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return torch.stack([_turn64(_norm64(x, s["q_weight"]), p.double(), case) for x, p in zip(s["x"], s["pos"])])
    ps, blk, table = case["ps"], case["blk"], s["table"].cpu().numpy()

    def place(b, first, count):
        at = np.arange(first, first + count)
        return torch.from_numpy(table[b][at // ps].astype(np.int64)).cuda(), torch.from_numpy(at % ps).cuda()

    def values(name, page, row):
        """Rows [n][Hkv][D] of a cache as numbers."""
        e = s[name + "_scale"][page, :, row // blk].int() - 127
        return s[name + "_cache"][page, :, row].double() * _two64(e)[..., None]

    if case["op"] == "read":
        out = {"k": s["k_out"].double(), "v": s["v_out"].double()}
        for b, n in enumerate(s["lens"]):
            for name in "kv":
                out[name][b, :, :n] = values(name, *place(b, 0, n)).transpose(0, 1)
        return out
    if case["op"] in ("append", "commit"):
        appends = case["op"] == "append"
        # block by block: with too many of them (some 20 s) the caches have no value here
        keep = sum(s["rows"]) // blk <= 8000 if appends else True
        par, dep = _parents(case) if appends and case["tree"] else (None, None)
        code = {n: s[n + "_cache"].double() for n in "kv"}
        exps = {n: s[n + "_scale"].int() - 127 for n in "kv"}
        was = {n: (code[n].clone(), exps[n].clone()) for n in "kv"}
        out = s["out"].double() if appends else None
        for b in range(case["B"]):
            P = s["lens"][b]
            if appends:
                n, first = s["rows"][b], P
                off = np.arange(n) if dep is None else dep[b, :n]
                pos = torch.from_numpy(P + off.astype(np.float64)).cuda()
                q, k = s["q"][b, :, :n].double(), s["k"][b, :, :n].double()
                if case["norm"]:
                    q, k = _norm64(q, s["q_weight"]), _norm64(k, s["k_weight"])
                out[b, :, :n] = _turn64(q, pos, case)
                fresh = {"k": _turn64(k, pos, case), "v": s["v"][b, :, :n].double()}  # [Hkv][n][D]
            else:
                path = [P + int(x) for x in s["accepted"][b]]
                n, first = len(path), P + 1
            if n == 0 or not keep:
                continue
            for b0 in range(first // blk * blk, first + n, blk):  # the blocks that receive rows
                lo, hi = max(b0, first), min(b0 + blk, first + n)
                page, r0 = int(table[b][b0 // ps]), b0 % ps
                for name in "kv":
                    c0, e0 = was[name]
                    old = e0[page, :, r0 // blk]
                    kept = c0[page, :, r0:r0 + lo - b0] * _two64(old)[:, None, None]
                    least = old if lo > b0 or not appends else torch.full_like(old, LEAST)
                    if appends:
                        rows = fresh[name][:, lo - first:hi - first]
                    else:
                        rows = []
                        for x in path[lo - first:hi - first]:
                            p, r = int(table[b][x // ps]), x % ps
                            e = e0[p, :, r // blk]
                            rows.append(c0[p, :, r] * _two64(e)[:, None])
                            least = torch.maximum(least, e)
                        rows = torch.stack(rows, 1)
                    new, e = _block_64(rows, least)
                    code[name][page, :, r0 + lo - b0:r0 + hi - b0] = new
                    code[name][page, :, r0:r0 + lo - b0] = _e4m3_64(kept * _two64(-e)[:, None, None])
                    exps[name][page, :, r0 // blk] = e
        got = {n + "_cache": code[n] if keep else None for n in "kv"}
        got |= {n + "_scale": _two64(exps[n]) if keep else None for n in "kv"}
        if appends:
            return got | {"q": out}
        new = torch.tensor([s["lens"][b] + len(p) + 1 for b, p in enumerate(s["accepted"])], dtype=torch.int32)
        return got | {"new_len": new}
    par, dep = _parents(case) if case["tree"] else (None, None)
    out = s["out"].double()
    G, D = case["Hq"] // case["Hkv"], case["D"]
    for b in range(case["B"]):
        n, P = s["rows"][b], s["lens"][b]
        hide = torch.zeros((n, P + n), dtype=torch.float64)
        hide[:, P:] = -math.inf
        depth = np.arange(n) if dep is None else dep[b, :n]
        if par is None:
            hide[:, P:] = torch.triu(hide[:, P:], 1)
        else:
            for i in range(n):
                a = i
                while a >= 0:
                    hide[i, P + a] = 0.0
                    a = int(par[b, a])
        where = torch.from_numpy(np.concatenate((np.arange(P), P + depth)).astype(np.float64))
        if case["window"]:
            hide[(where[P:, None] - where[None]) >= case["window"]] = -math.inf
        hide = hide.cuda()
        page, row = place(b, 0, P + n)
        kk, vv = values("k", page, row), values("v", page, row)
        for h in range(case["Hkv"]):
            k, v = kk[:, h], vv[:, h]
            for g in range(G):
                z = torch.einsum("id,jd->ij", s["q"][b, h * G + g, :n].double(), k) * D ** -0.5
                if case["cap"]:
                    z = torch.tanh(z / case["cap"]) * case["cap"]
                out[b, h * G + g, :n] = torch.softmax(z + hide, -1) @ v
    return out


def _seen(case):
    """(visible (row, key) pairs, distinct keys that some row sees) summed over the batch's sequences."""
    pairs = keys = 0
    dep_all = _parents(case)[1] if case["tree"] else None
    W = case["window"] or 1 << 40
    for b, (P, n) in enumerate(zip(_prefix(case), _rows(case))):
        dep = dep_all[b, :n].astype(np.int64) if case["tree"] else np.arange(n, dtype=np.int64)
        pairs += int((np.minimum(P, np.maximum(0, W - 1 - dep)) + np.minimum(dep + 1, W)).sum())
        keys += n + min(P, max(0, W - 1))
    return pairs, keys


def work(case):
    size = 2 if case.get("dtype", "bf16") == "bf16" else 4
    B, D = case["B"], case["D"]
    if case["op"] == "norm":
        n = B * case["H"] * case["N"]
        return {"bytes": 2 * n * D * size + 4 * B * case["N"] + D * size, "flops": n * (4 * D + 3 * case["rot"])}
    Hkv, blk = case["Hkv"], case["blk"]
    if case["op"] == "read":
        rows = sum(_prefix(case))
        return {"bytes": 2 * rows * Hkv * D * (1 + size) + 2 * rows * Hkv // blk + 4 * (rows // case["ps"] + B),
                "flops": 2 * rows * Hkv * D}
    if case["op"] == "commit":
        n = sum(case["L"] - b % (case["L"] // 2 + 1) for b in range(B))
        return {"bytes": 4 * n * Hkv * D + 4 * n + 12 * B, "flops": 0}
    Hq, rows = case["Hq"], sum(_rows(case))
    if case["op"] == "append":
        return {"bytes": rows * (Hq * D * 2 * size + 2 * Hkv * D * (size + 1)) + 2 * Hkv * (rows // blk + B) + 12 * B +
                (4 * B * case["N"] if case["tree"] else 0),
                "flops": rows * (Hq + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    pairs, keys = _seen(case)
    return {"bytes": 2 * keys * Hkv * D + 2 * keys * Hkv // blk + 2 * rows * Hq * D * size +
            4 * (keys // case["ps"] + B), "flops": 4 * D * Hq * pairs}
