"""CPU-side checks of the calls over 8-bit pages and of norms: host-side refusals of the C ABI and of
the binding (nothing is launched)."""
import ctypes
import math
import os
import shutil
import struct
import subprocess

import pytest

from test_abi import FAKE, NULL, lib  # noqa: F401  (the fixture builds a stale library)
from test_abi_paged import ODD, _Fake, _kv, _rope, _rows

torch = pytest.importorskip("torch")
E4M3 = torch.float8_e4m3fn


def _norm(q=0x1000, k=0x1000, eps=1e-6):
    from tree_speculative_decoding_masked_gb300 import _binding as b
    return b._pack_norm(q, k, eps)


def _scale(k=0x1001, v=0x1003, block=16):  # bytes: any address
    from tree_speculative_decoding_masked_gb300 import _binding as b
    return b._pack_scale(k, v, block)


def test_packed_structs_have_the_headers_layout(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "treeverify.h"\n'
                   'int main(void) { printf("%zu %zu %zu %zu\\n", sizeof(tv_head_norm), offsetof(tv_head_norm, eps),\n'
                   'sizeof(tv_kv_scale), offsetof(tv_kv_scale, block)); return 0; }\n')
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([gcc, "-I", inc, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [len(_norm()), 16, len(_scale()), 16]
    assert struct.unpack_from("@f", _norm(eps=0.5), 16) == (0.5,)
    assert struct.unpack_from("@i", _scale(block=8), 16) == (8,)


def test_norm_rotary_refusals(lib):  # noqa: F811
    def call(x=_rows(), out=FAKE, pos=FAKE, base=NULL, norm=_norm(k=0), rope=_rope(), B=1, H=1, N=1, D=64, dt=1):
        return lib.tv_norm_rotary(x, out, pos, base, norm, rope, B, H, N, D, dt, NULL)
    assert call(x=NULL) == -1 and call(x=_rows(data=0)) == -1 and call(out=NULL) == -1 and call(norm=NULL) == -1
    assert call(norm=_norm(q=0)) == -1 and call(pos=NULL) == -1 and call(rope=_rope(freq=0)) == -1
    assert call(dt=2) == -3 and call(dt=-1) == -3
    for bad in (dict(B=0), dict(H=0), dict(N=0), dict(D=0), dict(D=1025), dict(H=1 << 15), dict(rope=_rope(rot=66)),
                dict(rope=_rope(rot=3)), dict(B=1 << 16, N=1 << 16)):
        assert call(**bad) == -2, bad
    for eps in (-1.0, math.inf, math.nan):
        assert call(norm=_norm(eps=eps)) == -8
    assert call(rope=_rope(amp=math.nan)) == -8
    assert call(out=ODD) == -5 and call(x=_rows(data=0x1001)) == -5 and call(norm=_norm(q=0x1001)) == -5
    assert call(norm=_norm(q=0x1002), dt=0) == -5


def test_norm_append_refusals(lib):  # noqa: F811
    def call(k=_rows(), v=_rows(), kv=_kv(), norm=_norm(), rope=_rope(), q=_rows(), q_out=FAKE, B=1, Hq=2, Hkv=1, N=1,
             D=64, dt=1):
        return lib.tv_norm_append_kv_paged(k, v, kv, NULL, NULL, norm, rope, q, q_out, B, Hq, Hkv, N, D, dt, NULL, NULL)
    for bad in (dict(norm=NULL), dict(k=NULL), dict(v=NULL), dict(kv=NULL), dict(q_out=NULL), dict(norm=_norm(q=0)),
                dict(norm=_norm(k=0)), dict(kv=_kv(k=0)), dict(kv=_kv(prefix=0))):
        assert call(**bad) == -1, bad
    assert call(norm=_norm(eps=-1.0)) == -8 and call(norm=_norm(k=0x1001)) == -5
    assert call(Hq=0) == -2 and call(kv=_kv(ps=12)) == -2


def test_q8_append_refusals(lib):  # noqa: F811
    def call(k=_rows(), v=_rows(), kv=_kv(), scale=_scale(), norm=NULL, rope=_rope(), q=_rows(), q_out=FAKE, B=1, Hq=2,
             Hkv=1, N=1, D=64, dt=1):
        return lib.tv_append_kv_paged_q8(k, v, kv, scale, NULL, NULL, norm, rope, q, q_out, B, Hq, Hkv, N, D, dt, NULL,
                                         NULL)
    for bad in (dict(k=NULL), dict(v=NULL), dict(kv=NULL), dict(scale=NULL), dict(scale=_scale(k=0)),
                dict(scale=_scale(v=0)), dict(q_out=NULL), dict(rope=NULL), dict(norm=_norm(k=0)),
                dict(norm=_norm(q=0))):
        assert call(**bad) == -1, bad
    for bad in (dict(D=48), dict(D=288), dict(D=16), dict(scale=_scale(block=0)), dict(scale=_scale(block=3)),
                dict(scale=_scale(block=32)), dict(scale=_scale(block=128), kv=_kv(ps=128)), dict(scale=_scale(block=-1)),
                dict(B=65536), dict(kv=_kv(ps=4)), dict(N=0), dict(Hkv=0), dict(rope=_rope(rot=128))):
        assert call(**bad) == -2, bad
    assert call(dt=2) == -3
    assert call(norm=_norm(eps=math.nan)) == -8
    assert call(kv=_kv(k=0x1008)) == -5 and call(q_out=ODD) == -5 and call(k=_rows(data=0x1001)) == -5


def test_q8_read_refusals(lib):  # noqa: F811
    def call(kv=_kv(), scale=_scale(), k_out=FAKE, v_out=FAKE, B=1, Hkv=1, rows=4, D=64, dt=1):
        return lib.tv_read_kv_paged_q8(kv, scale, NULL, k_out, v_out, B, Hkv, rows, D, dt, NULL, NULL)
    for bad in (dict(kv=NULL), dict(scale=NULL), dict(k_out=NULL), dict(v_out=NULL), dict(scale=_scale(k=0))):
        assert call(**bad) == -1, bad
    for bad in (dict(rows=0), dict(rows=-1), dict(D=40), dict(B=0), dict(B=65536), dict(scale=_scale(block=64))):
        assert call(**bad) == -2, bad
    assert call(dt=5) == -3 and call(k_out=ctypes.c_void_p(0x1008)) == -5 and call(v_out=ODD) == -5


def test_q8_attention_refusals(lib):  # noqa: F811
    far = ctypes.c_void_p(0x100000)

    def call(q=FAKE, out=far, kv=_kv(), scale=_scale(), parent=NULL, B=1, Hq=2, Hkv=1, N=1, D=64, sc=0.0, cap=0.0,
             window=0, dt=1, ws=far, size=1 << 40):
        return lib.tv_paged_attention_q8(q, out, kv, scale, parent, NULL, B, Hq, Hkv, N, D, sc, cap, window, dt, ws, size,
                                         NULL, NULL)
    for bad in (dict(q=NULL), dict(out=NULL), dict(kv=NULL), dict(scale=NULL), dict(scale=_scale(v=0))):
        assert call(**bad) == -1, bad
    for bad in (dict(D=48), dict(D=320), dict(Hq=3, Hkv=2), dict(N=65537), dict(parent=FAKE, N=1025), dict(B=65536),
                dict(scale=_scale(block=5)), dict(scale=_scale(block=32))):
        assert call(**bad) == -2, bad
    for bad in (dict(sc=-1.0), dict(sc=math.nan), dict(cap=-1.0), dict(cap=math.inf), dict(window=-1), dict(out=FAKE)):
        assert call(**bad) == -8, bad
    assert call(dt=2) == -3 and call(q=ODD) == -5
    need = lib.tv_paged_attention_q8_workspace_size(64, 32, 8, 128, 64, 16, 64, 1)
    assert need > 0 and lib.tv_paged_attention_q8_workspace_size(1, 3, 2, 128, 1, 16, 64, 1) == 0
    assert call(B=64, Hq=32, Hkv=8, D=128, N=64, size=need - 1) == -4
    assert call(B=64, Hq=32, Hkv=8, D=128, N=64, ws=NULL) == -4


def test_q8_commit_refusals(lib):  # noqa: F811
    def call(kv=_kv(), scale=_scale(), nodes=FAKE, lens=FAKE, new=NULL, B=1, Hkv=1, N=4, D=64):
        return lib.tv_commit_accepted_kv_paged_q8(kv, scale, nodes, lens, new, B, Hkv, N, D, NULL, NULL)
    for bad in (dict(kv=NULL), dict(scale=NULL), dict(nodes=NULL), dict(lens=NULL)):
        assert call(**bad) == -1, bad
    for bad in (dict(N=1025), dict(N=0), dict(D=8), dict(scale=_scale(block=24))):
        assert call(**bad) == -2, bad
    assert call(new=FAKE) == -8


def _caches(**kw):
    pages = _Fake((4, 2, 16, 64), E4M3)
    a = dict(k_cache=pages, v_cache=_Fake((4, 2, 16, 64), E4M3), page_table=_Fake((1, 4), torch.int32),
             prefix_len=_Fake((1,), torch.int32), k_scale=_Fake((4, 2, 2), torch.uint8),
             v_scale=_Fake((4, 2, 2), torch.uint8))
    a.update(kw)
    return a


BAD_SCALES = [
    (dict(k_scale=None), "need k_scale"),
    (dict(v_scale=None), "need k_scale"),
    (dict(k_scale=_Fake((4, 2, 2), torch.float32)), "uint8 or"),
    (dict(k_scale=_Fake((4, 2), torch.uint8)), "uint8 or"),
    (dict(k_scale=_Fake((4, 2, 3), torch.uint8)), "3 blocks a page"),
    (dict(k_scale=_Fake((4, 2, 0), torch.uint8)), "0 blocks a page"),
    (dict(k_scale=_Fake((3, 2, 2), torch.uint8)), "must have shape"),
    (dict(v_scale=_Fake((4, 2, 1), torch.uint8)), "must have shape"),
    (dict(v_scale=_Fake((4, 2, 2), torch.float8_e8m0fnu)), "must be torch.uint8"),
    (dict(v_scale=_Fake((4, 2, 2), torch.uint8, stride=(8, 4, 2))), "contiguous"),
    (dict(k_cache=_Fake((4, 2, 16, 64)), v_cache=_Fake((4, 2, 16, 64))), "belong to caches of"),
]


@pytest.mark.parametrize("bad,match", BAD_SCALES)
def test_binding_refuses_scales(bad, match):
    import tree_speculative_decoding_masked_gb300 as tv
    rows, q = _Fake((1, 2, 3, 64)), _Fake((1, 4, 3, 64))
    nodes = dict(accepted_nodes=_Fake((1, 4), torch.int32), accept_len=_Fake((1,), torch.int32))
    out = _Fake((1, 4, 3, 64))
    status = _Fake((1,), torch.int32)
    with pytest.raises(ValueError, match=match):
        tv.append_kv_paged(rows, rows, **_caches(**bad))
    with pytest.raises(ValueError, match=match):
        tv.paged_attention(q, **_caches(**bad), out=out, workspace=_Fake((8,), torch.uint8), dev_status=status)
    with pytest.raises(ValueError, match=match):
        tv.commit_accepted_kv_paged(**_caches(**bad), **nodes, new_len=_Fake((1,), torch.int32), dev_status=status)
    a = _caches(**bad)
    a["length"] = a.pop("prefix_len")
    with pytest.raises(ValueError, match=match):
        tv.read_kv_paged(**a, k_out=rows, v_out=rows)


def test_binding_refuses_norms_and_rows():
    import tree_speculative_decoding_masked_gb300 as tv
    x, w, pos = _Fake((1, 2, 3, 64)), _Fake((64,)), _Fake((1, 3), torch.int32)
    rope = {"freq": _Fake((32,), torch.int64), "rot_dim": 64, "amplitude": 1.0}
    for bad, match in ((_Fake((32,)), "must have shape"), (_Fake((64,), torch.float32), "must be torch.bfloat16")):
        with pytest.raises(ValueError, match=match):
            tv.norm_rotary(x, bad, pos, rope, out=x)
        with pytest.raises(ValueError, match=match):
            tv.append_kv_paged(x, x, **_caches(), norm=(None, bad, 1e-6), dev_status=_Fake((1,), torch.int32))
    with pytest.raises(ValueError, match="pos is required"):
        tv.norm_rotary(x, w, None, rope, out=x)
    with pytest.raises(TypeError, match="unsupported dtype"):
        tv.norm_rotary(_Fake((1, 2, 3, 64), torch.float16), w, pos, rope)
    with pytest.raises(ValueError, match="rope is required"):
        tv.append_kv_paged(x, x, **_caches(), q=x)
    with pytest.raises(TypeError, match="unsupported dtype"):
        tv.append_kv_paged(_Fake((1, 2, 3, 64), torch.float16), x, **_caches())
    a = _caches(k_cache=_Fake((4, 2, 16, 64)), v_cache=_Fake((4, 2, 16, 64)), k_scale=None, v_scale=None)
    a["length"] = a.pop("prefix_len")
    with pytest.raises(ValueError, match="reads caches of"):
        tv.read_kv_paged(**a)
    a = _caches()
    a["length"] = a.pop("prefix_len")
    with pytest.raises(ValueError, match="v_out must have shape"):
        tv.read_kv_paged(**a, k_out=_Fake((1, 2, 5, 64)), v_out=_Fake((1, 2, 6, 64)))
