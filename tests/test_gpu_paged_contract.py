"""GPU tests of what the header promises for calls over pages beside their results."""
import pytest

import synth
from test_gpu_paged import _status

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import tree_speculative_decoding_masked_gb300 as tv  # noqa: E402
from gpu_util import dev, i32, to_dev  # noqa: E402


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
