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


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad,good", [([0, 40, 10, 60], [0, 40, 40, 60]),
                                      ([0, 60, 0, 60, 0, 60], [0] + [60] * 5),
                                      ([70, 5, -3, 10 ** 9, 40], [60] * 5)])
def test_a_row_has_one_group_whatever_the_offsets(bad, good, dtype):
    """Offsets that turn back: an offset below an earlier one counts as the
    earlier one, so that no row is written twice and the tiles are bounded by
    the rows (1024 groups that turn back over 2^20 rows, 32768 features: 2^31
    tiles of 64 x 128, more than their 32-bit numbers hold)."""
    G, n, k = len(bad) - 1, 96, 128
    x, w = R.normal(1, 60, k, dtype=dtype), R.normal(2, G, n, k, dtype=dtype, std=k ** -0.5)
    dy = R.normal(3, 60, n, dtype=dtype)
    a = moe.checkpoint_rows(R.normal(4, 60, k, dtype=dtype).cuda())
    for call in (lambda o, s: [moe.grouped_linear(x.cuda(), w.cuda(), o, status=s)],
                 lambda o, s: [moe.grouped_linear_dx(dy.cuda(), w.cuda(), o, status=s)],
                 lambda o, s: [moe.swiglu_checkpoint(x.cuda(), w.cuda(), w.cuda(), o, status=s)[0]],
                 lambda o, s: moe.swiglu_backward(dy.cuda(), w.cuda(), a, a, o, status=s)):
        s1, s2 = status(), status()
        got, want = call(offs(bad), s1), call(offs(good), s2)
        assert int(s1.item()) == -6 and int(s2.item()) == 0
        for t, v in zip(got, want):
            assert torch.equal(t[good[0]:good[-1]], v[good[0]:good[-1]])


# wide, narrow and split tiles of the staged fp32 products
STAGED = [([300, 900], 640, 1032), ([70, 0, 90], 640, 1100), ([700], 96, 2500)]


@pytest.mark.parametrize("sizes,n,k", STAGED)
def test_largest_finite_fp32_operands(sizes, n, k):
    """Magnitudes between bf16's largest value and fp32's, which a first bf16
    term would round to infinity, in the rows and in the weights."""
    off, top = R.offsets_of(sizes), torch.finfo(F32).max
    rows, G = off[-1], len(sizes)
    assert float(torch.tensor(top).to(BF)) == float("inf")
    x, dy = R.normal(1, rows, k, dtype=F32), R.normal(2, rows, n, dtype=F32)
    w = R.normal(3, G, n, k, dtype=F32, std=2.0 ** -20)
    x[60, 5], x[7, 0], x[60, 9] = 3.4e38, -top, 3.3962e38   # two of them in one sum: below 2^108 each
    w[0, 11, 3], dy[7, 2] = top, -3.4e38
    x[:, 3] *= 2.0 ** -20
    dy[:, 11] *= 2.0 ** -20
    st = status()
    y = moe.grouped_linear(x.cuda(), w.cuda(), offs(off), status=st)
    R.assert_close(y, *R.linear(x, w, off), "linear")
    d = moe.grouped_linear_dx(dy.cuda(), w.cuda(), offs(off), status=st)
    R.assert_close(d, *R.dx(dy, w, off), "dx")
    xs = R.normal(4, rows, k, dtype=F32, std=2.0 ** -20)
    R.assert_close(moe.grouped_linear_dw(dy.cuda(), xs.cuda(), offs(off), status=st), *R.dw(dy, xs, off), "dw")
    w *= 2.0 ** -90                          # projections of at most 2^20 or so
    h, *_ = moe.swiglu_checkpoint(x.cuda(), w.cuda(), w.cuda(), offs(off), status=st)
    assert torch.isfinite(h).all()
    assert int(st.item()) == 0


@pytest.mark.parametrize("sizes,n,k", STAGED)
def test_smallest_fp32_operands(sizes, n, k):
    """Operand bits below 2^-133 are lost, half a step of them at most a value."""
    off = R.offsets_of(sizes)
    x, w = R.normal(1, off[-1], k, dtype=F32), R.normal(2, len(sizes), n, k, dtype=F32)
    x *= torch.exp2(torch.linspace(-135, -100, off[-1]))[:, None]
    y = moe.grouped_linear(x.cuda(), w.cuda(), offs(off))
    v, e = R.linear(x, w, off)
    lost = R.linear(torch.ones_like(x), w.abs(), off)[0] * 2.0 ** -134
    R.assert_close(y, v, e + 1.01 * lost)
