"""The kernels that serve the training operators' large cases: tiles of SM
pairs, several of them a pair, their stage rings wrapped many times, with empty
and short groups among the long ones.  Whole results against 64-bit forms."""
import pytest
import torch

import train_ref as R
import sparse_moe_layer_sum_b200 as moe

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_moe_layer_sum_b200 import build
    build.build_all()


def offs(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("out", [BF, F32])
def test_dw_of_long_groups_that_end_inside_a_step(dtype, out):
    """Many blocks that need no zeroing before the one that does."""
    sizes, n, k = [1501, 0, 2047, 33, 1], 1100 if dtype == BF else 600, 1032
    off = R.offsets_of(sizes)
    dy, x = R.normal(1, off[-1], n, dtype=dtype), R.normal(2, off[-1], k, dtype=dtype)
    st = status()
    got = moe.grouped_linear_dw(dy.cuda(), x.cuda(), offs(off), out_dtype=out, status=st)
    assert int(st.item()) == 0
    R.assert_close(got, *R.dw(dy, x, off))
    again = moe.grouped_linear_dw(dy.cuda(), x.cuda(), offs(off), out_dtype=out)
    assert torch.equal(got, again)
