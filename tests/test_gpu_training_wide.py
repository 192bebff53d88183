"""The kernels that serve the training operators' large cases: tiles of SM
pairs, several of them a pair, their stage rings wrapped many times, with empty
and short groups among the long ones.  Whole results against 64-bit forms."""
import pytest
import torch

import test_gpu_experts_training as step
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


# Shapes for which every product takes the tiles of SM pairs (several pairs have
# more than one of them), partial tiles of rows and of features, groups of none,
# of a row and of less than a tile, and contractions that wrap the stage rings
# many times.  The third is past 64 k-blocks, where backward's first segments
# are twice as long; its fp32 operands have six times as many.
WIDE = [([700, 0, 900, 33, 65, 130], 1304, 1096),
        ([257, 513, 1, 700, 0, 300, 255], 2056, 584),
        ([600, 0, 410, 1, 300], 1544, 4232),
        ([700, 0, 900, 33, 65, 130], 1301, 1099)]   # off the pitch: through padded copies


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes,n,k", WIDE)
def test_wide_products(sizes, n, k, dtype, out):
    off = R.offsets_of(sizes, first=2)
    rows, G = off[-1] + 3, len(sizes)
    x, dy, dy2 = (R.normal(i, rows, c, dtype=dtype) for i, c in ((1, k), (2, n), (3, n)))
    w, w2 = (R.normal(i, G, n, k, dtype=dtype, std=k ** -0.5) for i in (4, 5))
    xd, dyd, dy2d, wd, w2d = (t.cuda() for t in (x, dy, dy2, w, w2))
    o, st = offs(off), status()
    live = slice(off[0], off[-1])
    y = torch.full((rows, n), 7.0, dtype=out, device="cuda")
    d = torch.full((rows, k), 7.0, dtype=out, device="cuda")
    for got, (want, e), what in (
            (moe.grouped_linear(xd, wd, o, out=y, status=st), R.linear(x, w, off), "linear"),
            (moe.grouped_linear_dx(dyd, wd, o, out=d, status=st), R.dx(dy, w, off), "dx"),
            (moe.grouped_linear_dx(dyd, wd, o, dy2=dy2d, w2=w2d, out_dtype=out, status=st),
             R.dx(dy, w, off, dy2, w2), "dx of two")):
        R.assert_close(got[live], want[live], e[live], what)
    for t in (y, d):                                     # rows of no group
        assert (t[:off[0]] == 7.0).all() and (t[off[-1]:] == 7.0).all()
    R.assert_close(moe.grouped_linear_dw(dyd, xd, o, out_dtype=out, status=st), *R.dw(dy, x, off), "dw")
    assert int(st.item()) == 0


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes,n,k", WIDE)
def test_wide_swiglu_backward(sizes, n, k, dtype, gated):
    off = R.offsets_of(sizes)
    rows, G = off[-1], len(sizes)
    dy = R.normal(1, rows, k, dtype=dtype)
    w2 = R.normal(2, G, k, n, dtype=dtype, std=n ** -0.5)
    a, u = (moe.checkpoint_rows(R.normal(i, rows, n, dtype=F32, std=2.0).cuda()) for i in (3, 4))
    gate = torch.rand(rows, generator=torch.Generator().manual_seed(5)) + 0.1
    st = status()
    got = moe.swiglu_backward(dy.cuda(), w2.cuda(), a, u, offs(off), gate=gate.cuda() if gated else None,
                              status=st)
    assert int(st.item()) == 0
    dh, e = R.dx(dy, w2, off)
    av, uv = (R.decode(c.codes.cpu(), c.exps.cpu()) for c in (a, u))
    gate = gate if gated else torch.ones_like(gate)
    vals, errs = R.swiglu_grads(av, uv, dh, e, gate.to(R.F64), dtype)
    for g, v, b, name in zip(got, vals, errs, ("da", "du", "hg", "dgate")):
        R.assert_close(g, v, b, name)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_wide_swiglu_checkpoint(dtype):
    sizes, n, k = WIDE[2]
    off = R.offsets_of(sizes)
    x = R.normal(1, off[-1], k, dtype=dtype)
    w1, w3 = (R.normal(i, len(sizes), n, k, dtype=dtype, std=2 * k ** -0.5) for i in (2, 3))
    h, a, u = moe.swiglu_checkpoint(x.cuda(), w1.cuda(), w3.cuda(), offs(off))
    (av, ae), (uv, ue) = R.linear(x, w1, off), R.linear(x, w3, off)
    s = R.silu(av).abs()
    err = 1.1 * ae * (uv.abs() + ue) + s * ue + s * uv.abs() * (R.sigmoid_rel(av, dtype) + 4 * R.ULP)
    R.assert_close(h, R.silu(av) * uv, err, "h")
    for c, v, e in ((a, av, ae), (u, uv, ue)):
        exps = c.exps.cpu()
        scale = torch.exp2(exps.to(R.F64) - 127).repeat_interleave(32, 1)[:, :n]
        # half a step of a code: 2^-4 of the value, or 2^-10 of the scale
        d = (R.decode(c.codes.cpu(), exps) - v).abs()
        assert (d <= torch.maximum(2.0 ** -4 * (v.abs() + e), scale * 2.0 ** -10) + e).all()


def test_wide_shapes_take_the_wide_tiles():
    """What train.cu's wide() asks, for each product of WIDE and of the step
    below: rows a group on average, and tiles for half the 74 SM pairs."""
    for sizes, n, k in WIDE:
        rows, G = sum(sizes), len(sizes)
        assert rows / G > 48
        # (features, rows of a tile, features of one) of linear, dx and backward
        for F, bn, feat in ((n, 256, 512), (k, 256, 512), (n, 256, 256), (k, 256, 256), (n, 128, 256)):
            if F == 584 and feat == 512:
                continue                      # dx to 584: narrow tiles in bf16
            assert (rows // bn + min(rows, G)) * -(-F // feat) >= 37, (sizes, F, bn, feat)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_wide_step(dtype):
    """The experts' forward and backward pass with about 360 rows a group."""
    step.test_forward_and_backward(dict(T=600, dtype=dtype, dim=1032, inter=1304, n_routed=4, n_groups=1,
                                        topk_groups=1, topk=2))


def test_threads_with_inputs_of_their_own():
    """Calls at once from several threads and streams, each on other inputs and
    sizes: a workspace or a plan that two of them shared would show."""
    import threading
    torch.cuda.synchronize()

    def inputs(i):
        sizes, n, k = [[70, 0, 131, 5], [300, 41, 0, 9], [64, 64, 1, 700], [5, 3, 0, 90]][i], 264 + 8 * i, 520
        off = R.offsets_of(sizes)
        rows, G, dt = off[-1], len(sizes), F32 if i % 2 else BF
        t = dict(x=R.normal(10 * i, rows, k, dtype=dt), dy=R.normal(10 * i + 1, rows, k, dtype=dt),
                 w1=R.normal(10 * i + 2, G, n, k, dtype=dt, std=k ** -0.5),
                 w3=R.normal(10 * i + 3, G, n, k, dtype=dt, std=k ** -0.5),
                 w2=R.normal(10 * i + 4, G, k, n, dtype=dt, std=n ** -0.5))
        return {a: b.cuda() for a, b in t.items()} | {"off": offs(off)}

    def work(t):
        h, a, u = moe.swiglu_checkpoint(t["x"], t["w1"], t["w3"], t["off"])
        y = moe.grouped_linear(h, t["w2"], t["off"])
        da, du, hg, dgate = moe.swiglu_backward(t["dy"], t["w2"], a, u, t["off"])
        dx = moe.grouped_linear_dx(da, t["w1"], t["off"], dy2=du, w2=t["w3"])
        return [h, a.codes, u.exps, y, da, du, hg, dgate, dx, moe.grouped_linear_dw(da, t["x"], t["off"]),
                moe.grouped_linear_dw(t["dy"], hg, t["off"])]

    each = [inputs(i) for i in range(4)]
    want = [work(t) for t in each]
    torch.cuda.synchronize()
    same = [None] * 4

    def loop(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [work(each[i]) for _ in range(10)]
        s.synchronize()
        same[i] = all(torch.equal(a, b) for g in got for a, b in zip(g, want[i]))

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert same == [True] * 4
