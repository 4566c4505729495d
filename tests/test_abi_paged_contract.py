"""CPU-side checks of the paged calls' refusals: outputs that lie over what the kernels read meanwhile
(nothing is launched)."""
import ctypes

from test_abi import NULL, lib  # noqa: F401  (the fixture builds a stale library)
from test_abi_paged import _kv


def test_new_len_may_not_lie_over_what_the_commit_reads(lib):  # noqa: F811
    B, N, width = 3, 5, 4
    at = dict(prefix=0x11000, table=0x12000, acc=0x13000, n=0x14000)
    size = dict(prefix=4 * B, table=4 * B * width, acc=4 * B * N, n=4 * B)

    def call(new):
        return lib.tv_commit_accepted_kv_paged(_kv(prefix=at["prefix"], table=at["table"], width=width),
                                               ctypes.c_void_p(at["acc"]), ctypes.c_void_p(at["n"]), ctypes.c_void_p(new),
                                               B, 2, N, 64, 1, NULL, NULL)
    for name, start in at.items():
        for new in (start, start + 4, start - 4, start - 4 * B + 4, start + size[name] - 4):
            assert call(new) == -8, (name, hex(new))


def test_attentions_output_may_not_lie_over_its_queries(lib):  # noqa: F811
    B, Hq, N, D = 2, 4, 3, 64
    q = 0x100000
    for dt, size in ((0, 4 * B * Hq * N * D), (1, 2 * B * Hq * N * D)):
        for out in (q, q + 16, q - 16, q + size - 16, q - size + 16):
            assert lib.tv_paged_attention(ctypes.c_void_p(q), ctypes.c_void_p(out), _kv(), NULL, NULL, B, Hq, 2, N, D, 0.0,
                                          0.0, 0, dt, ctypes.c_void_p(0x200000), 1 << 40, NULL, NULL) == -8
