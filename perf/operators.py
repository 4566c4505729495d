"""Timing cases of the paged verification round: rotary positions, the append of keys and
values to a paged cache, attention over it, and the commit of an accepted path.

Each case runs either in a plain form (elementary torch operations in 32 bits, angles in
64) or, with ``own`` true, through the framework's calls.  ``exact`` states every operator
once more in 64 bits.

Shapes follow the repository's synthetic workloads (32 query and 8 KV heads of 128, trees of
16 to 1024 nodes, prefixes to 32768) and the single-token and prompt-chunk steps around a
verification round.  Caches hold pages in random order, as a server's free list leaves them,
and the sequences of a batch have different lengths.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the queries of one 64-node tree, far into a stretched context: latency
        dict(name="rotary_tree", op="rotary", B=1, H=32, N=64, D=128, rot=128, inter=False, scaling="yarn", P=120000,
             dtype="bf16"),
        # a prompt chunk's queries, interleaved pairs over half of the head: bandwidth
        dict(name="rotary_chunk", op="rotary", B=4, H=32, N=4096, D=128, rot=64, inter=True, scaling="linear", P=8192,
             dtype="bf16"),
        # one token of a small batch, queries rotated in the same call: latency
        dict(name="append_token", op="append", B=4, Hq=32, Hkv=8, N=1, D=128, ps=16, P=2048, rot=128, inter=False,
             scaling="none", tree=False, dtype="bf16"),
        # ragged prompt chunks with their queries: bandwidth
        dict(name="append_chunk", op="append", B=4, Hq=32, Hkv=8, N=2048, D=128, ps=32, P=4001, rot=128, inter=False,
             scaling="banded", tree=False, dtype="bf16"),
        # one sequence, one token: latency
        dict(name="attend_token", op="attend", B=1, Hq=32, Hkv=8, N=1, D=128, ps=16, P=2048, tree=False, cap=0.0,
             window=0, dtype="bf16"),
        # a full decoding batch of ragged lengths: bandwidth
        dict(name="attend_batch", op="attend", B=64, Hq=32, Hkv=8, N=1, D=128, ps=16, P=16384, tree=False, cap=0.0,
             window=0, dtype="bf16"),
        # the single-layer workload's 64-node tree over pages
        dict(name="attend_tree", op="attend", B=1, Hq=32, Hkv=8, N=64, D=128, ps=16, P=2048, tree=True, cap=0.0,
             window=0, dtype="bf16"),
        # the long-context workload's trees over pages, lengths ragged
        dict(name="attend_tree_long", op="attend", B=8, Hq=32, Hkv=8, N=128, D=128, ps=64, P=32768, tree=True, cap=0.0,
             window=0, dtype="bf16"),
        # prompt chunks behind a prefix, causal
        dict(name="attend_chunk", op="attend", B=2, Hq=32, Hkv=8, N=2048, D=128, ps=32, P=6000, tree=False, cap=0.0,
             window=0, dtype="bf16"),
        # capped scores and a sliding window, 32-bit, odd sizes
        dict(name="attend_cap_f32", op="attend", B=2, Hq=8, Hkv=4, N=100, D=64, ps=16, P=3001, tree=True, cap=30.0,
             window=1024, dtype="f32"),
        # one sequence's accepted path
        dict(name="commit_tree", op="commit", B=1, Hkv=8, N=64, D=128, ps=16, P=2048, L=5, dtype="bf16"),
        # a full batch's accepted paths
        dict(name="commit_batch", op="commit", B=64, Hkv=8, N=256, D=128, ps=16, P=4096, L=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attend", "attend", "attend", "commit"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([64, 128, 128])
    ps = rng.choice([8, 16, 32, 64, 128])
    scaling = rng.choice(["none", "linear", "base", "banded", "yarn"])
    if op == "rotary":
        N = _log(rng, 1, 4096)
        return dict(op=op, B=max(1, min(_log(rng, 1, 32), 16384 // N)), H=rng.choice([8, 16, 32]), N=N, D=D,
                    rot=rng.choice([D, D // 2, 32]), inter=rng.random() < 0.5, scaling=scaling, P=_log(rng, 1, 500000),
                    dtype=dtype)
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    if op == "append":
        tree = rng.random() < 0.5
        N = _log(rng, 1, 256 if tree else 2048)
        return dict(op=op, B=max(1, min(_log(rng, 1, 64), 8192 // N)), Hq=Hq, Hkv=Hkv, N=N, D=D, ps=ps,
                    P=_log(rng, 1, 4000), rot=rng.choice([D, D // 2]), inter=rng.random() < 0.5, scaling=scaling,
                    tree=tree, dtype=dtype)
    if op == "commit":
        N = _log(rng, 16, 1024)
        return dict(op=op, B=_log(rng, 1, 64), Hkv=Hkv, N=N, D=D, ps=ps, P=_log(rng, 1, 4000),
                    L=rng.randint(0, min(16, N // 2 - 1)), dtype=dtype)
    kind = rng.choice(["token", "tree", "chunk"])
    N = 1 if kind == "token" else _log(rng, 2, 512) if kind == "tree" else _log(rng, 2, 2048)
    P = _log(rng, 1, 24000)
    # the score count (an eighth of it in 32 bits, which run on CUDA cores) and the cache of the largest listed cases
    # bound B
    wide = dtype == "f32"
    most, cache = 8 * 32 * 128 * 32768 // (8 if wide else 1), 64 * 12288 * 8 * 128 // (2 if wide else 1)
    B = max(1, min(_log(rng, 1, 64), most // (Hq * N * (P + N)), cache // ((P + N) * Hkv * D)))
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, N=N, D=D, ps=ps, P=P, tree=kind == "tree",
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


_SCALING = {"none": None, "linear": ("linear", 4.0), "base": ("base", 4.0), "banded": ("banded", 8.0, 1.0, 4.0, 8192),
            "yarn": ("yarn", 16.0, 8192, 32.0, 1.0)}
_BASE = 500000.0


def _inv_freq(rot, scaling):
    """Rotary frequencies (radians a position, float64) and the amplitude of the rotated part."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = _BASE ** (-i / rot)
    s = _SCALING[scaling]
    if s is None:
        return f, 1.0
    if s[0] == "linear":
        return f / s[1], 1.0
    if s[0] == "base":
        return (_BASE * s[1] ** (rot / (rot - 2.0))) ** (-i / rot), 1.0
    if s[0] == "banded":
        _, factor, lo, hi, length = s
        mix = ((length * f / (2 * math.pi) - lo) / (hi - lo)).clamp(0.0, 1.0)
        return f * (mix + (1 - mix) / factor), 1.0
    _, factor, length, fast, slow = s

    def dim(turns):
        return rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(_BASE))
    lo, hi = max(math.floor(dim(fast)), 0), min(math.ceil(dim(slow)), rot - 1)
    keep = 1 - ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0


def _randn(shape, gen, dtype):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // max(1, math.prod(shape[1:])))
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        out[i:i + n] = torch.randn((n, *shape[1:]), generator=gen, device="cuda", dtype=torch.float32)
    return out


def _ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _paged(case, gen):
    """A cache of just the pages that the batch needs and a few more, and the table of each sequence's pages."""
    B, ps = case["B"], case["ps"]
    need = [(p + case["N"] + ps - 1) // ps for p in _prefix(case)]
    width, pages = max(need) + 1, sum(need) + 5
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    shape = (pages, case["Hkv"], ps, case["D"])
    return _randn(shape, gen, DTYPES[case["dtype"]]), _randn(shape, gen, DTYPES[case["dtype"]]), table


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, s = DTYPES[case["dtype"]], dict(case=case)
    if case["op"] in ("rotary", "append"):
        f, amp = _inv_freq(case["rot"], case["scaling"])
        s["inv_freq"], s["amp"] = f.cuda(), amp
        if own:
            import tree_speculative_decoding_masked_gb300 as tv
            s["rope"] = tv.rotary_frequencies(case["rot"], _BASE, scaling=_SCALING[case["scaling"]], device="cuda")
    s["dev_status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] == "rotary":
        B, H, N, D = (case[k] for k in "BHND")
        # token-major rows, as a projection writes them
        s["x"] = _randn((B, N, H, D), gen, dt).transpose(1, 2)
        start = torch.randint(0, case["P"], (B, 1), generator=gen, device="cuda", dtype=torch.int32)
        s["pos"] = (start + torch.arange(N, device="cuda", dtype=torch.int32)).contiguous()
        s["out"] = torch.zeros((B, H, N, D), dtype=dt, device="cuda")
        return s
    B, Hkv, N, D = case["B"], case["Hkv"], case["N"], case["D"]
    s["lens"], s["rows"] = _prefix(case), _rows(case)
    s["k_cache"], s["v_cache"], s["table"] = _paged(case, gen)
    s["prefix_len"], s["n_rows"] = _ints(s["lens"]), _ints(s["rows"])
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
        n = tv.paged_attention_workspace_size(B, Hq, Hkv, D, N, case["ps"], s["table"].shape[1], dt)
        s["workspace"] = torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")
    return s


# ---- plain forms


def _rotate(x, pos, s):
    """x [B][H][N][D] at positions pos [B][N] (float64 angles), the product in 32 bits."""
    case, rot = s["case"], s["case"]["rot"]
    ang = pos.double()[:, None, :, None] * s["inv_freq"]
    cos, sin = (ang.cos() * s["amp"]).float(), (ang.sin() * s["amp"]).float()
    y = x.float().clone()
    if case["inter"]:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y.to(x.dtype)


def _places(s):
    """(sequence, new row, page, row in the page) of every active new row."""
    t = torch.arange(s["case"]["N"], device="cuda", dtype=torch.int64)
    b, t = torch.nonzero(t[None] < s["n_rows"][:, None], as_tuple=True)
    at = s["prefix_len"].long()[b] + t
    return b, t, s["table"].long()[b, at // s["case"]["ps"]], at % s["case"]["ps"]


def _plain_append(s):
    case = s["case"]
    off = torch.arange(case["N"], device="cuda")[None] if s["depth"] is None else s["depth"]
    pos = s["prefix_len"][:, None] + off
    b, t, page, row = _places(s)
    s["k_cache"][page, :, row] = _rotate(s["k"], pos, s)[b, :, t]
    s["v_cache"][page, :, row] = s["v"][b, :, t]
    s["out"][b, :, t] = _rotate(s["q"], pos, s)[b, :, t]
    return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


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
        j = torch.arange((max(s["lens"][b0:b0 + n]) + N + ps - 1) // ps * ps, device="cuda")
        L = j.numel()
        pages = s["table"][b0:b0 + n, :L // ps].clamp(min=0).long()
        k, v = (s[c][pages].permute(0, 2, 1, 3, 4).reshape(n, Hkv, L, D).float() for c in ("k_cache", "v_cache"))
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
        q = s["q"][b0:b0 + n].float().reshape(n, Hkv, G, N, D)
        z = q.reshape(n, Hkv, G * N, D) @ k.transpose(-1, -2) / math.sqrt(D)
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
    case, P = s["case"], s["prefix_len"].long()
    k = torch.arange(case["N"], device="cuda")
    b, k = torch.nonzero(k[None] < s["accept_len"][:, None], as_tuple=True)
    src, dst = P[b] + s["accepted_nodes"].long()[b, k], P[b] + k + 1
    table, ps = s["table"].long(), case["ps"]
    for c in (s["k_cache"], s["v_cache"]):
        c[table[b, dst // ps], :, dst % ps] = c[table[b, src // ps], :, src % ps]
    s["new_len"].copy_(s["prefix_len"] + s["accept_len"] + 1)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "new_len": s["new_len"]}


def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        if op == "rotary":
            s["out"].copy_(_rotate(s["x"], s["pos"], s))
            return s["out"]
        return {"append": _plain_append, "attend": _plain_attend, "commit": _plain_commit}[op](s)
    import tree_speculative_decoding_masked_gb300 as tv
    if op == "rotary":
        return tv.rotary(s["x"], s["pos"], s["rope"], interleaved=case["inter"], out=s["out"])
    if op == "append":
        tv.append_kv_paged(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], depth=s["depth"],
                           n_rows=s["n_rows"], rope=s["rope"], interleaved=case["inter"], q=s["q"], q_out=s["out"],
                           dev_status=s["dev_status"])
        return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "commit":
        tv.commit_accepted_kv_paged(s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], s["accepted_nodes"],
                                    s["accept_len"], new_len=s["new_len"], dev_status=s["dev_status"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "new_len": s["new_len"]}
    return tv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], parent=s["parent"],
                              n_rows=s["n_rows"], softcap=case["cap"], window=case["window"], out=s["out"],
                              workspace=s["workspace"], dev_status=s["dev_status"])


# ---- 64-bit statement


def _turn64(x, pos, case):
    """One row set x [..., D] (float64) turned by complex products; pos broadcasts over the leading axes."""
    rot = case["rot"]
    f, amp = _inv_freq(rot, case["scaling"])
    w = torch.polar(torch.full_like(pos[..., None] * f.to(x.device), amp), pos[..., None] * f.to(x.device))
    head = x[..., :rot]
    pair = head.unflatten(-1, (rot // 2, 2)) if case["inter"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    y = torch.view_as_real(torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * w)
    y = y.flatten(-2) if case["inter"] else y.transpose(-1, -2).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return torch.stack([_turn64(x.double(), p.double(), case) for x, p in zip(s["x"], s["pos"])])
    ps, table = case["ps"], s["table"].cpu().numpy()

    def place(b, first, count):
        at = np.arange(first, first + count)
        return torch.from_numpy(table[b][at // ps].astype(np.int64)).cuda(), torch.from_numpy(at % ps).cuda()

    if case["op"] == "commit":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for c in (kc, vc):
            old = c.clone()
            for b, path in enumerate(s["accepted"]):
                for k, a in enumerate(path):
                    i, j = s["lens"][b] + int(a), s["lens"][b] + k + 1
                    c[table[b][j // ps], :, j % ps] = old[table[b][i // ps], :, i % ps]
        new = torch.tensor([s["lens"][b] + len(p) + 1 for b, p in enumerate(s["accepted"])], dtype=torch.int32)
        return {"k_cache": kc, "v_cache": vc, "new_len": new}
    par, dep = _parents(case) if case["tree"] else (None, None)
    if case["op"] == "append":
        kc, vc, out = s["k_cache"].double(), s["v_cache"].double(), s["out"].double()
        for b in range(case["B"]):
            n, P = s["rows"][b], s["lens"][b]
            if n == 0:
                continue
            off = np.arange(n) if dep is None else dep[b, :n]
            pos = torch.from_numpy(P + off.astype(np.float64)).cuda()
            page, row = place(b, P, n)
            kc[page, :, row] = _turn64(s["k"][b, :, :n].double(), pos, case).transpose(0, 1)
            vc[page, :, row] = s["v"][b, :, :n].double().transpose(0, 1)
            out[b, :, :n] = _turn64(s["q"][b, :, :n].double(), pos, case)
        return {"q": out, "k_cache": kc, "v_cache": vc}
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
        for h in range(case["Hkv"]):
            k, v = s["k_cache"][page, h, row].double(), s["v_cache"][page, h, row].double()
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
    size = 2 if case["dtype"] == "bf16" else 4
    B, N, D = case["B"], case["N"], case["D"]
    if case["op"] == "rotary":
        n = B * case["H"] * N
        return {"bytes": 2 * n * D * size + 4 * B * N, "flops": 3 * n * case["rot"]}
    if case["op"] == "commit":
        n = sum(case["L"] - b % (case["L"] // 2 + 1) for b in range(B))
        return {"bytes": 4 * n * (case["Hkv"] * D * size + 1) + 12 * B, "flops": 0}
    Hq, Hkv, rows = case["Hq"], case["Hkv"], sum(_rows(case))
    if case["op"] == "append":
        return {"bytes": 2 * rows * (Hq + 2 * Hkv) * D * size + 12 * B + (4 * B * N if case["tree"] else 0),
                "flops": 3 * rows * (Hq + Hkv) * case["rot"]}
    pairs, keys = _seen(case)
    return {"bytes": 2 * keys * Hkv * D * size + 2 * rows * Hq * D * size + 4 * (keys // case["ps"] + B),
            "flops": 4 * D * Hq * pairs}
