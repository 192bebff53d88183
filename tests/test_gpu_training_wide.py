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


def positive(seed, rows, cols, by):
    """Positive values, each row or column (by: 0, 1) with a magnitude of its
    own, so that long sums of them lie anywhere between two bf16 values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.rand(rows, cols, generator=g, device="cuda", dtype=F32).add_(0.5)
    m = torch.rand((rows, 1) if by == 0 else (1, cols), generator=g, device="cuda").add_(1.0)
    return v.mul_(m).to(BF)


def assert_rounded(got, want, cut):
    """bf16 results of long sums of one sign: roundings to nearest (2^-8)
    average out, to 2^-8 / sqrt(n) or so; what the sums are cut by does not.
    cut: how much that may be, on average and at most."""
    rel = (got.double() - want) / want
    assert rel.abs().max() <= 2.0 ** -8 * (1 + cut) + cut
    assert got.numel() > 2 ** 17 and rel.mean().abs() < cut


# in segments of 512 values: 32 cuts by at most 2^-23 of the sum each, and 2^9
# fp32 additions to nearest; in one go up to 2^16 values: 2^12 such cuts
SEGMENTS, WHOLE = 2.0 ** -14, 2.0 ** -11


@pytest.mark.parametrize("rows,F", [(640, 1024), (4096, 2048)])    # narrow and wide tiles
def test_long_contractions_round_once(rows, F):
    k = 1 << 17
    x, w = positive(1, rows, k, 0), positive(2, F, k, 0)[None]
    want = x.double() @ w[0].double().T
    assert_rounded(moe.grouped_linear(x, w, offs([0, rows])), want, SEGMENTS)
    w = w.transpose(1, 2).contiguous()
    assert_rounded(moe.grouped_linear_dx(x, w, offs([0, rows])), want, SEGMENTS)
    # of two products, each within the length that one may have
    h = k // 2
    a, b = x[:, :h].contiguous(), x[:, h:].contiguous()
    got = moe.grouped_linear_dx(a, w[:, :h].contiguous(), offs([0, rows]), dy2=b, w2=w[:, h:].contiguous())
    assert_rounded(got, want, SEGMENTS)


@pytest.mark.parametrize("n,accumulate", [(1600, False), (1600, True), (200, False)])
def test_dw_of_very_long_groups_rounds_once(n, accumulate):
    """Long groups between short and empty ones; a length at the border."""
    sizes, k = [300, 0, 200001, 1 << 16, 77], 1536 if n > 256 else 1544
    off = R.offsets_of(sizes)
    dy, x = positive(1, off[-1], n, 1), positive(2, off[-1], k, 1)
    st = status()
    base = torch.ones(len(sizes), n, k, dtype=BF, device="cuda")
    got = moe.grouped_linear_dw(dy, x, offs(off), out=base.clone(), accumulate=accumulate, status=st)
    for g, r in R.groups(off):
        want = dy[r].double().T @ x[r].double() + float(accumulate)
        if r.stop - r.start > 300:
            assert_rounded(got[g], want, SEGMENTS if g == 2 else WHOLE)
        else:
            e = (r.stop - r.start + 2) * R.ULP * want
            R.assert_close(got[g], want.cpu(), e.cpu())
    assert int(st.item()) == 0


def test_results_over_their_operands_are_refused():
    x, w = R.normal(1, 40, 64).cuda(), R.normal(2, 2, 64, 64).cuda()
    o, dw = offs([0, 20, 40]), torch.zeros(2, 64, 64, dtype=BF, device="cuda")
    both = torch.zeros(80, 64, dtype=BF, device="cuda")
    codes = both.view(torch.uint8).view(-1)[:40 * 64].view(40, 64)
    exps = torch.zeros(40, 2, dtype=torch.uint8, device="cuda")
    for call in (lambda: moe.grouped_linear(x, w, o, out=x),
                 lambda: moe.grouped_linear(both[1:41], w, o, out=both[40:]),
                 lambda: moe.grouped_linear_dx(x, w, o, out=x),
                 lambda: moe.grouped_linear_dx(x, w, o, dy2=both[:40], w2=w, out=both[39:79]),
                 lambda: moe.grouped_linear_dw(dw[0], dw[1], offs([0, 30, 64]), out=dw),
                 lambda: moe.restore_rows(moe.Checkpoint(codes, exps), out=both[:40])):
        with pytest.raises(ValueError, match="share memory"):
            call()
    # side by side is fine
    assert moe.grouped_linear(both[:40], w, o, out=both[40:]).data_ptr() == both[40:].data_ptr()
    assert moe.restore_rows(moe.Checkpoint(codes, exps), out=both[40:]).shape == (40, 64)
