"""CPU-side checks of the paged calls and rotary positions: host-side refusals of the C ABI
and of the binding (nothing is launched), and the frequencies, which are made on the host."""
import ctypes
import math

import numpy as np
import pytest

from oracle import rotary
from test_abi import FAKE, NULL, lib  # noqa: F401  (the fixture builds a stale library)

torch = pytest.importorskip("torch")
ODD = ctypes.c_void_p(0x1001)


class _Fake:
    """Stands in for a CUDA tensor (nothing is launched)."""

    def __init__(self, shape, dtype=torch.bfloat16, device="cpu", stride=None, ptr=0x1000):
        self.shape, self.dtype, self.is_cuda, self.device = tuple(shape), dtype, True, torch.device(device)
        dense = [math.prod(shape[i + 1:]) for i in range(len(shape))]
        self.ndim = len(shape)
        self._stride, self._dense, self._ptr = tuple(stride or dense), tuple(dense), ptr

    def is_contiguous(self):
        return self._stride == self._dense

    def stride(self):
        return self._stride

    def get_device(self):
        return self.device.index or 0

    def data_ptr(self):
        return self._ptr

    def numel(self):
        return math.prod(self.shape)

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()


def _rows(data=0x1000, strides=(64, 64, 64)):
    from tree_speculative_decoding_masked_gb300 import _binding as b
    return b._pack_rows(data or 0, *strides)


def _rope(freq=0x1000, rot=64, amp=1.0):
    from tree_speculative_decoding_masked_gb300 import _binding as b
    return b._pack_rope(freq or 0, rot, 0, amp)


def _kv(k=0x1000, v=0x1000, table=0x1000, prefix=0x1000, pages=4, ps=16, width=4):
    from tree_speculative_decoding_masked_gb300 import _binding as b
    return b._pack_paged_kv(k or 0, v or 0, table or 0, prefix or 0, pages, ps, width)


def test_packed_structs_have_the_headers_layout(tmp_path):
    # sizes and offsets of the host structs, asked of the C compiler
    import os
    import shutil
    import struct
    import subprocess
    from tree_speculative_decoding_masked_gb300 import _binding as b
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "treeverify.h"\n'
                   'int main(void) { printf("%zu %zu %zu %zu %zu %zu %zu\\n", sizeof(tv_rope), offsetof(tv_rope, amplitude),\n'
                   'sizeof(tv_rows), offsetof(tv_rows, row_stride), sizeof(tv_paged_kv), offsetof(tv_paged_kv, prefix_len),\n'
                   'offsetof(tv_paged_kv, max_pages)); return 0; }\n')
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([gcc, "-I", inc, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [len(_rope()), 16, len(_rows()), 24, len(_kv()), 24, 40]
    assert struct.unpack_from("@f", _rope(amp=2.5), 16) == (2.5,)
    assert struct.unpack_from("@q", b._pack_rows(1, 2, 3, 4), 24) == (4,)
    assert struct.unpack_from("@iii", _kv(pages=5, ps=8, width=7), 32) == (5, 8, 7)


def test_frequencies(lib):  # noqa: F811
    import tree_speculative_decoding_masked_gb300 as tv
    for scaling in (None, ("linear", 4.0), ("base", 8.0), ("banded", 8.0, 1.0, 4.0, 8192),
                    ("yarn", 16.0, 4096, 32.0, 1.0)):
        for rot in (4, 20, 64, 128):
            got = tv.rotary_frequencies(rot, 500000.0, scaling=scaling, device="cpu")
            ref, amp = rotary.frequencies(rot, 500000.0, scaling)
            turns = got["freq"].numpy().view(np.uint64).astype(np.float64) * 2.0 ** -64
            # half a step of 2^-62 turns, and a few roundings of 64-bit floats
            assert np.all(np.abs(turns - ref / (2 * math.pi)) <= 2.0 ** -62 + 2.0 ** -49 * turns)
            assert abs(got["amplitude"] - amp) <= 2.0 ** -23 and got["rot_dim"] == rot
    with pytest.raises(ValueError, match="unknown scaling"):
        tv.rotary_frequencies(64, scaling=("dynamic", 2.0), device="cpu")
    with pytest.raises(ValueError, match="takes 4 parameters"):
        tv.rotary_frequencies(64, scaling=("yarn", 2.0), device="cpu")


def test_frequency_refusals(lib):  # noqa: F811
    f = lib.tv_rotary_frequencies
    out, amp = (ctypes.c_uint64 * 64)(), ctypes.c_float()

    def call(rot=64, base=1e4, kind=0, params=(), dst=out, a=ctypes.byref(amp)):
        return f(rot, base, kind, (ctypes.c_double * 4)(*params) if params else NULL, dst, a)
    assert call() == 0
    assert call(dst=NULL) == -1 and call(a=NULL) == -1 and call(kind=1) == -1
    for rot in (0, 1, 63, -2, 1026):
        assert call(rot=rot) == -2
    assert call(rot=2, kind=2, params=(2,)) == -2
    for base in (1.0, 0.0, -3.0, math.inf, math.nan):
        assert call(base=base) == -8
    for kind, params in ((-1, ()), (5, ()), (1, (0.5,)), (1, (math.nan,)), (3, (2, 4, 4, 100)), (3, (2, 1, 4, 0)),
                         (3, (2, 1, 4, math.inf)), (4, (2, 0, 32, 1)), (4, (2, 100, 1, 32)), (4, (2, 100, 32, 0))):
        assert call(kind=kind, params=params) == -8, (kind, params)


def test_rotary_and_append_refusals(lib):  # noqa: F811
    def rot(x=_rows(), out=FAKE, pos=FAKE, rope=_rope(), B=1, H=2, N=3, D=64, dt=1):
        return lib.tv_rotary(x, out, pos, NULL, rope, B, H, N, D, dt, NULL)
    assert rot(x=NULL) == rot(x=_rows(None)) == rot(out=NULL) == rot(pos=NULL) == rot(rope=NULL) == -1
    assert rot(rope=_rope(None)) == -1
    assert rot(dt=2) == -3
    for kw in (dict(B=0), dict(H=0), dict(N=0), dict(D=0), dict(D=1025), dict(rope=_rope(rot=66)),
               dict(rope=_rope(rot=7)), dict(rope=_rope(rot=-2)), dict(B=1 << 20, N=1 << 20)):
        assert rot(**kw) == -2, kw
    assert rot(rope=_rope(amp=math.inf)) == rot(rope=_rope(amp=math.nan)) == -8
    assert rot(x=_rows(0x1001)) == rot(out=ODD) == -5
    assert rot(x=_rows(0x1002), dt=0) == -5

    def app(k=_rows(), v=_rows(), kv=_kv(), rope=_rope(), q=NULL, qo=NULL, B=1, Hq=4, Hkv=2, N=3, D=64, dt=1):
        return lib.tv_append_kv_paged(k, v, kv, NULL, NULL, rope, q, qo, B, Hq, Hkv, N, D, dt, NULL, NULL)
    assert app(k=NULL) == app(v=_rows(None)) == app(kv=NULL) == -1
    assert app(kv=_kv(k=None)) == app(kv=_kv(table=None)) == app(kv=_kv(prefix=None)) == -1
    assert app(q=_rows()) == app(q=_rows(), qo=FAKE, rope=NULL) == app(q=_rows(None), qo=FAKE) == -1
    assert app(dt=9) == -3
    for kw in (dict(kv=_kv(ps=4)), dict(kv=_kv(ps=24)), dict(kv=_kv(ps=2048)), dict(kv=_kv(pages=0)),
               dict(kv=_kv(width=0)), dict(kv=_kv(width=1 << 28)), dict(kv=_kv(width=(1 << 26) + 1)), dict(kv=_kv(pages=1 << 30), Hkv=4), dict(N=0),
               dict(q=_rows(), qo=FAKE, Hq=0), dict(rope=_rope(rot=128))):
        assert app(**kw) == -2, kw
    assert app(kv=_kv(k=0x1008)) == app(kv=_kv(v=0x1004)) == app(D=12, rope=NULL) == app(k=_rows(0x1001)) == -5
    assert app(q=_rows(0x1001), qo=FAKE) == app(q=_rows(), qo=ODD) == -5


def test_attention_and_commit_refusals(lib):  # noqa: F811
    size = lib.tv_paged_attention_workspace_size
    assert size(0, 4, 2, 64, 1, 16, 4, 1) == size(1, 3, 2, 64, 1, 16, 4, 1) == size(1, 4, 2, 40, 1, 16, 4, 1) == 0
    big = 1 << 40

    def att(q=FAKE, out=FAKE, kv=_kv(), par=NULL, B=1, Hq=4, Hkv=2, N=3, D=64, scale=0.0, cap=0.0, win=0, dt=1,
            ws=FAKE, n=big):
        return lib.tv_paged_attention(q, out, kv, par, NULL, B, Hq, Hkv, N, D, scale, cap, win, dt, ws, n, NULL, NULL)
    assert att(q=NULL) == att(out=NULL) == att(kv=NULL) == att(kv=_kv(v=None)) == -1
    assert att(dt=5) == -3
    for kw in (dict(Hq=3), dict(Hq=0), dict(D=48), dict(D=288), dict(N=65537), dict(par=FAKE, N=1025),
               dict(kv=_kv(ps=12)), dict(Hq=2048, N=65536)):
        assert att(**kw) == -2, kw
    for kw in (dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(cap=-1.0), dict(cap=math.nan),
               dict(cap=math.inf), dict(win=-1), dict(cap=1e-45), dict(scale=1e30, cap=1e-20)):
        assert att(**kw) == -8, kw
    assert att(q=ODD) == att(out=ctypes.c_void_p(0x1008)) == att(kv=_kv(k=0x1004)) == -5
    need = size(1, 4, 2, 64, 3, 16, 4, 0)
    if need:
        assert att(ws=NULL, dt=0) == att(n=need - 1, dt=0) == -4
        assert att(ws=ctypes.c_void_p(0x1008), dt=0) == -5

    def com(kv=_kv(), acc=FAKE, n=FAKE, new=NULL, B=1, Hkv=2, N=3, D=64, dt=1):
        return lib.tv_commit_accepted_kv_paged(kv, acc, n, new, B, Hkv, N, D, dt, NULL, NULL)
    assert com(kv=NULL) == com(acc=NULL) == com(n=NULL) == -1
    assert com(dt=4) == -3 and com(N=1025) == com(B=65536) == com(Hkv=0) == -2
    assert com(D=12) == com(kv=_kv(k=0x1001)) == -5
    assert com(new=FAKE) == -8  # prefix_len itself


def test_binding_refusals(lib):  # noqa: F811
    import tree_speculative_decoding_masked_gb300 as tv
    i32, f32 = torch.int32, torch.float32
    rope = {"freq": _Fake((32,), torch.int64), "amplitude": 1.0, "rot_dim": 64}
    x, pos = _Fake((2, 4, 3, 64)), _Fake((2, 3), i32)

    def refuse(match, f, *a, **kw):
        with pytest.raises((ValueError, TypeError), match=match):
            f(*a, **kw)
    refuse("CUDA", tv.rotary, x, torch.zeros((2, 3), dtype=i32), rope)
    refuse("CUDA", tv.rotary, torch.zeros((2, 4, 3, 64), dtype=torch.bfloat16), pos, rope)
    refuse("pos must have shape", tv.rotary, x, _Fake((2, 4), i32), rope)
    refuse("pos must be torch.int32", tv.rotary, x, _Fake((2, 3), torch.int64), rope)
    refuse("pos_base must have shape", tv.rotary, x, pos, rope, pos_base=_Fake((3,), i32))
    refuse("unsupported dtype", tv.rotary, _Fake((2, 4, 3, 64), torch.float16), pos, rope)
    refuse("last dimension", tv.rotary, _Fake((2, 4, 3, 64), stride=(768, 192, 1, 3)), pos, rope)
    refuse("out must have shape", tv.rotary, x, pos, rope, out=_Fake((2, 4, 3, 32)))
    refuse("out must be torch.bfloat16", tv.rotary, x, pos, rope, out=_Fake((2, 4, 3, 64), f32))
    refuse("contiguous to be rotated in place", tv.rotary, _Fake((2, 4, 3, 64), stride=(768, 64, 256, 1)), pos, rope,
           out=x)
    refuse("freq", tv.rotary, x, pos, dict(rope, rot_dim=32))
    refuse("one device", tv.rotary, _Fake((2, 4, 3, 64), device="cuda:1"), pos, rope)
    kc, table, pre = _Fake((9, 2, 16, 64)), _Fake((2, 4), i32), _Fake((2,), i32)
    k = _Fake((2, 2, 3, 64))
    refuse("k_cache and v_cache", tv.append_kv_paged, k, k, kc, _Fake((9, 2, 8, 64)), table, pre)
    refuse("must be contiguous", tv.append_kv_paged, k, k, kc,
           _Fake((9, 2, 16, 64), stride=(2048, 64, 128, 1)), table, pre)
    refuse("one device", tv.append_kv_paged, k, k, kc, _Fake((9, 2, 16, 64), device="cuda:1"), table, pre)
    refuse("CUDA", tv.append_kv_paged, k, k, kc, torch.zeros((9, 2, 16, 64), dtype=torch.bfloat16), table, pre)
    refuse("k must have shape", tv.append_kv_paged, _Fake((2, 3, 3, 64)), k, kc, kc, table, pre)
    refuse("v must have shape", tv.append_kv_paged, k, _Fake((2, 2, 4, 64)), kc, kc, table, pre)
    refuse("v must be torch.bfloat16", tv.append_kv_paged, k, _Fake((2, 2, 3, 64), f32), kc, kc, table, pre)
    refuse("page_table must be torch.int32", tv.append_kv_paged, k, k, kc, kc, _Fake((2, 4), torch.int64), pre)
    refuse("prefix_len must have shape", tv.append_kv_paged, k, k, kc, kc, table, _Fake((3,), i32))
    refuse("depth must have shape", tv.append_kv_paged, k, k, kc, kc, table, pre, depth=_Fake((2, 4), i32))
    refuse("n_rows must be", tv.append_kv_paged, k, k, kc, kc, table, pre, n_rows=_Fake((2,), f32))
    refuse("rope is required", tv.append_kv_paged, k, k, kc, kc, table, pre, q=x)
    refuse("q must have shape", tv.append_kv_paged, k, k, kc, kc, table, pre, q=_Fake((2, 4, 5, 64)), rope=rope)
    refuse("q_out must have shape", tv.append_kv_paged, k, k, kc, kc, table, pre, q=x, q_out=k, rope=rope)
    refuse("q must have shape", tv.paged_attention, _Fake((3, 4, 3, 64)), kc, kc, table, pre)
    refuse("q must be torch.bfloat16", tv.paged_attention, _Fake((2, 4, 3, 64), f32), kc, kc, table, pre)
    refuse("must be contiguous", tv.paged_attention, _Fake((2, 4, 3, 64), stride=(768, 64, 256, 1)), kc, kc, table,
           pre)
    refuse("parent must have shape", tv.paged_attention, x, kc, kc, table, pre, parent=_Fake((2, 4), i32))
    refuse("n_rows must have shape", tv.paged_attention, x, kc, kc, table, pre, n_rows=_Fake((2, 1), i32))
    refuse("out must have shape", tv.paged_attention, x, kc, kc, table, pre, out=k)
    refuse("accepted_nodes must be", tv.commit_accepted_kv_paged, kc, kc, table, pre, _Fake((2, 5), torch.int64), pre)
    refuse("accept_len must have shape", tv.commit_accepted_kv_paged, kc, kc, table, pre, _Fake((2, 5), i32),
           _Fake((3,), i32))
    refuse("new_len must be", tv.commit_accepted_kv_paged, kc, kc, table, pre, _Fake((2, 5), i32), pre,
           new_len=_Fake((2,), f32))


def test_attention_output_and_workspace_refusals(lib):  # noqa: F811
    import tree_speculative_decoding_masked_gb300 as tv
    for dt in (0, 1):  # q itself: other CTAs may still read it
        assert lib.tv_paged_attention(FAKE, FAKE, _kv(), NULL, NULL, 1, 4, 2, 3, 64, 0.0, 0.0, 0, dt,
                                      ctypes.c_void_p(0x2000), 1 << 40, NULL, NULL) == -8
    x, kc, table, pre = _Fake((2, 4, 3, 64)), _Fake((9, 2, 16, 64)), _Fake((2, 4), torch.int32), _Fake((2,), torch.int32)
    # an expanded workspace holds fewer bytes than its elements count
    ws = _Fake((1 << 30,), torch.uint8, stride=(0,))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        tv.paged_attention(x, kc, kc, table, pre, out=_Fake((2, 4, 3, 64), ptr=0x9000), workspace=ws,
                           dev_status=_Fake((1,), torch.int32))
