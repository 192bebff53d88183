"""The experts' training operators against 64-bit CPU forms."""
import pytest
import torch

import train_ref as R
import sparse_moe_layer_sum_b200 as moe

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# (sizes of the groups, n, k): rows of one and of none, groups off and across
# every tile, widths off every alignment and widths with partial tiles
SHAPES = [
    ([1], 8, 8),
    ([0, 3, 0, 1, 0], 64, 128),
    ([16, 17, 31, 64, 65], 128, 256),
    ([130, 0, 257, 1], 136, 200),
    ([300, 12, 513], 520, 264),
    ([5, 40, 2], 33, 77),
    ([1, 2], 1, 1),
    ([700], 640, 576),
    # large enough for the tensor cores although off their alignment
    ([300, 0, 513, 1, 17], 333, 301),
    ([21, 33, 90, 40, 64, 15, 77, 8, 130, 1], 607, 449),
    ([700, 0, 900, 33], 607, 537),
    ([700, 0, 900, 33], 640, 520),
    # few tiles with a long contraction, which is cut into parts
    ([5, 0, 40], 96, 2504),
    ([3], 2056, 72),
    ([0, 2900, 1800], 72, 64),
    ([900, 6], 100, 1302),
]


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_moe_layer_sum_b200 import build
    build.build_all()


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def offs(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes,n,k", SHAPES)
def test_products(sizes, n, k, dtype):
    off = R.offsets_of(sizes)
    rows, G = off[-1], len(sizes)
    x, dy, dy2 = (R.normal(i, rows, c, dtype=dtype) for i, c in ((1, k), (2, n), (3, n)))
    w, w2 = (R.normal(i, G, n, k, dtype=dtype, std=k ** -0.5) for i in (4, 5))
    xd, dyd, dy2d, wd, w2d = dev(x, dy, dy2, w, w2)
    o, st = offs(off), status()
    for out in (BF, F32):
        y = moe.grouped_linear(xd, wd, o, out_dtype=out, status=st)
        assert y.dtype == out
        R.assert_close(y, *R.linear(x, w, off), "linear")
        R.assert_close(moe.grouped_linear_dx(dyd, wd, o, out_dtype=out, status=st),
                       *R.dx(dy, w, off), "dx")
        R.assert_close(moe.grouped_linear_dx(dyd, wd, o, dy2=dy2d, w2=w2d, out_dtype=out, status=st),
                       *R.dx(dy, w, off, dy2, w2), "dx of two")
        R.assert_close(moe.grouped_linear_dw(dyd, xd, o, out_dtype=out, status=st),
                       *R.dw(dy, x, off), "dw")
        base = R.normal(6, G, n, k, dtype=out)
        acc = base.cuda()
        moe.grouped_linear_dw(dyd, xd, o, out=acc, accumulate=True, status=st)
        v, e = R.dw(dy, x, off)
        want = v + base.to(R.F64)
        # one more fp32 addition, of magnitude at most |base| + sum |terms|
        R.assert_close(acc, want, 2 * e + R.ULP * (base.to(R.F64).abs() + v.abs()), "dw accumulated")
        for g, s in enumerate(sizes):
            if s == 0:
                assert torch.equal(acc[g].cpu(), base[g])
    assert int(st.item()) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,k,sizes", [(128, 256, [21, 0, 70, 9]), (520, 264, [21, 0, 70, 9]),
                                       (33, 77, [21, 0, 70, 9]), (520, 264, [210, 0, 700, 90]),
                                       (607, 449, [210, 0, 700, 90]), (40, 1600, [21, 0, 70, 9])])
def test_rows_outside_the_groups_stay(n, k, sizes, dtype):
    """Rows before the first and behind the last group are left as they were,
    and what they hold (NaN here) reaches no result; neither does a NaN in
    another group's rows or weights."""
    off = R.offsets_of(sizes, first=3)
    rows, G = off[-1] + 40, 4
    x, dy = R.normal(1, rows, k, dtype=dtype), R.normal(2, rows, n, dtype=dtype)
    w = R.normal(3, G, n, k, dtype=dtype, std=k ** -0.5)
    nan = float("nan")
    bad_x, bad_dy, bad_w = x.clone(), dy.clone(), w.clone()
    for t in (bad_x, bad_dy):
        t[:off[0]] = nan
        t[off[-1]:] = nan
        t[off[2]:off[3]] = nan          # all of group 2
    bad_w[1], bad_w[2] = nan, float("inf")
    live = torch.zeros(rows, dtype=torch.bool)
    live[off[0]:off[2]] = True
    live[off[3]:off[4]] = True
    out = torch.zeros(rows, dtype=torch.bool)
    out[:off[0]] = out[off[-1]:] = True
    xd, dyd, wd, o = bad_x.cuda(), bad_dy.cuda(), bad_w.cuda(), offs(off)
    y = torch.full((rows, n), 7.0, dtype=dtype, device="cuda")
    moe.grouped_linear(xd, wd, o, out=y)
    d = torch.full((rows, k), 7.0, dtype=dtype, device="cuda")
    moe.grouped_linear_dx(dyd, wd, o, out=d)
    g = moe.grouped_linear_dw(dyd, xd, o)
    for got, (want, e) in ((y, R.linear(x, w, off)), (d, R.dx(dy, w, off))):
        assert (got[out.cuda()] == 7.0).all()
        R.assert_close(got[live.cuda()], want[live], e[live])
    want, e = R.dw(dy, x, off)
    keep = [0, 1, 3]
    R.assert_close(g[keep], want[keep], e[keep])
    assert torch.isnan(g[2]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_groups(dtype):
    """The most groups there can be, most of them empty or of a row or two."""
    G, n, k = 1024, 64, 72
    g = torch.Generator().manual_seed(4)
    sizes = torch.randint(-6, 5, (G,), generator=g).clamp_min(0).tolist()
    sizes[17], sizes[1023] = 130, 70
    off = R.offsets_of(sizes)
    x, dy = R.normal(1, off[-1], k, dtype=dtype), R.normal(2, off[-1], n, dtype=dtype)
    w = R.normal(3, G, n, k, dtype=dtype)
    xd, dyd, wd = dev(x, dy, w)
    o, st = offs(off), status()
    R.assert_close(moe.grouped_linear(xd, wd, o, status=st), *R.linear(x, w, off))
    R.assert_close(moe.grouped_linear_dx(dyd, wd, o, status=st), *R.dx(dy, w, off))
    R.assert_close(moe.grouped_linear_dw(dyd, xd, o, status=st), *R.dw(dy, x, off))
    h, a, u = moe.swiglu_checkpoint(xd, wd, wd, o, status=st)
    got = moe.swiglu_backward(xd, wd.transpose(1, 2).contiguous(), a, u, o, status=st)
    assert int(st.item()) == 0
    dh, e = R.dx(x, w.transpose(1, 2), off)
    av, uv = (R.decode(c.codes.cpu(), c.exps.cpu()) for c in (a, u))
    for t, v, b in zip(got, *R.swiglu_grads(av, uv, dh, e, torch.ones(off[-1], dtype=R.F64), dtype)):
        R.assert_close(t, v, b)


def shifted(t):
    """t's values at an address one element off a fresh allocation's."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    v = buf[1:].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes,n,k", [([5, 70], 64, 128), ([300, 0, 290], 520, 328)])
def test_misaligned_operands(sizes, n, k, dtype):
    off = R.offsets_of(sizes)
    rows, G = off[-1], len(sizes)
    x, dy = R.normal(1, rows, k, dtype=dtype), R.normal(2, rows, n, dtype=dtype)
    w = R.normal(3, G, n, k, dtype=dtype, std=k ** -0.5)
    xd, dyd, wd = shifted(x), shifted(dy), shifted(w)
    o = offs(off)
    y = shifted(torch.zeros(rows, n, dtype=dtype))
    R.assert_close(moe.grouped_linear(xd, wd, o, out=y), *R.linear(x, w, off))
    R.assert_close(moe.grouped_linear_dx(dyd, wd, o), *R.dx(dy, w, off))
    g = shifted(torch.zeros(G, n, k, dtype=dtype))
    R.assert_close(moe.grouped_linear_dw(dyd, xd, o, out=g), *R.dw(dy, x, off))
    # results at odd addresses from aligned operands
    R.assert_close(moe.grouped_linear(x.cuda(), w.cuda(), o, out=y), *R.linear(x, w, off))
    R.assert_close(moe.grouped_linear_dw(dy.cuda(), x.cuda(), o, out=g), *R.dw(dy, x, off))
    h, a, u = moe.swiglu_checkpoint(xd, wd, wd, o)
    want = moe.swiglu_checkpoint(x.cuda(), w.cuda(), w.cuda(), o)
    R.assert_close(h, want[0].cpu().to(R.F64), 2 * R.HALF[dtype] * want[0].cpu().to(R.F64).abs() +
                   1e-5)  # two roundings, and two sums of unit-variance terms
    a = moe.Checkpoint(shifted(a.codes), shifted(a.exps))
    w2 = R.normal(4, G, k, n, dtype=dtype, std=n ** -0.5)
    got = moe.swiglu_backward(xd, shifted(w2), a, u, o)
    dh, e = R.dx(x, w2, off)
    av, uv = (R.decode(c.codes.cpu(), c.exps.cpu()) for c in (a, u))
    for t, v, b in zip(got, *R.swiglu_grads(av, uv, dh, e, torch.ones(rows, dtype=R.F64), dtype)):
        R.assert_close(t, v, b)


def test_results_past_32_bit_offsets():
    """More than 2^31 elements in a result; the rows around that mark."""
    n, k, rows = 8192, 64, 270000
    x, w = R.normal(1, 3000, k), R.normal(2, 3, n, k, std=k ** -0.5)
    off = [0, 1000, 262000, rows]
    idx = (torch.arange(rows) % 3000).int()
    xd, wd = moe.gather_rows(x.cuda(), idx.cuda()), w.cuda()
    y = moe.grouped_linear(xd, wd, offs(off))
    at = torch.tensor([0, 999, 1000, 261999, 262000, 262143, 262144, 262145, rows - 1])
    assert rows * n > 2 ** 31 and (262144 * n == 2 ** 31)
    for i in at.tolist():
        g = sum(i >= o for o in off) - 1
        v, e = R.linear(x[idx[i].long()][None], w[g][None], [0, 1])
        R.assert_close(y[i][None], v, e, f"row {i}")
    c = moe.checkpoint_rows(y)
    r = moe.restore_rows(c)
    exps = R.scale_exps(y[at.cuda()].cpu())
    assert torch.equal(c.exps[at.cuda()].cpu(), exps)
    assert torch.equal(r[at.cuda()].cpu().to(R.F64), R.decode(c.codes[at.cuda()].cpu(), exps))
    del c, r
    dxr = moe.grouped_linear_dx(y, wd, offs(off))             # reads past the mark
    for i in at.tolist()[-3:]:
        v, e = R.dx(y[i][None].cpu(), w[2][None], [0, 1])
        R.assert_close(dxr[i][None], v, e, f"dx row {i}")
    del y, dxr
    # a weight gradient with its last matrices past the mark
    G, n, k = 33, 8192, 8192
    dy, x = R.normal(3, 99, n), R.normal(4, 99, k)
    dw = moe.grouped_linear_dw(dy.cuda(), x.cuda(), offs([3 * g for g in range(G + 1)]))
    assert dw.numel() > 2 ** 31
    for g in (0, 31, 32):
        v, e = R.dw(dy[3 * g:3 * g + 3], x[3 * g:3 * g + 3], [0, 3])
        R.assert_close(dw[g, -300:, -300:][None], v[:, -300:, -300:], e[:, -300:, -300:])


@pytest.mark.parametrize("dtype,sizes", [(BF, [300, 0, 513, 1, 17]), (F32, [300, 0, 513, 1, 17]),
                                         (F32, [400, 3, 700, 0, 17])])
def test_without_a_workspace(dtype, sizes):
    """The C entry points without a workspace: the CUDA cores do it."""
    import ctypes
    from sparse_moe_layer_sum_b200._lib import MoEGroupedShape, fn
    n, k = 333, 301
    off = R.offsets_of(sizes)
    rows, G = off[-1], len(sizes)
    x, dy = R.normal(1, rows, k, dtype=dtype), R.normal(2, rows, n, dtype=dtype)
    w = R.normal(3, G, n, k, dtype=dtype, std=k ** -0.5)
    xd, dyd, wd = dev(x, dy, w)
    o, dt = offs(off), int(dtype == BF)
    s = ctypes.byref(MoEGroupedShape(G, n, k, rows))
    if dtype == BF or rows > 1000:  # sizes for which one is asked for
        assert fn("moe_train", "moe_grouped_linear_workspace_size")(s, dt, 1) > 0
    stream = torch.cuda.current_stream().cuda_stream
    y, d, g = (torch.empty(*t, dtype=dtype, device="cuda") for t in ((rows, n), (rows, k), (G, n, k)))
    assert fn("moe_train", "moe_grouped_linear")(s, xd.data_ptr(), dt, wd.data_ptr(), o.data_ptr(),
                                                 y.data_ptr(), dt, None, 0, None, stream) == 0
    assert fn("moe_train", "moe_grouped_linear_dx")(s, dyd.data_ptr(), dt, wd.data_ptr(), None, None,
                                                    o.data_ptr(), d.data_ptr(), dt, None, 0, None,
                                                    stream) == 0
    assert fn("moe_train", "moe_grouped_linear_dw")(s, dyd.data_ptr(), dt, xd.data_ptr(), o.data_ptr(),
                                                    g.data_ptr(), dt, 0, None, 0, None, stream) == 0
    R.assert_close(y, *R.linear(x, w, off))
    R.assert_close(d, *R.dx(dy, w, off))
    R.assert_close(g, *R.dw(dy, x, off))


def test_infinite_operands_stay_in_their_rows():
    """fp32 operands in three terms: rows that meet an infinity are not finite,
    the others are as without it."""
    off = R.offsets_of([300, 500])
    x, w = R.normal(1, 800, 520, dtype=F32), R.normal(2, 2, 640, 520, dtype=F32)
    bad = x.clone()
    bad[7, 3], bad[401, 0], bad[500, 519] = float("inf"), float("-inf"), float("nan")
    bad[600, 5] = 3.4e38                     # rounds to infinity in bf16, but is not
    y = moe.grouped_linear(bad.cuda(), w.cuda(), offs(off)).cpu()
    hit = torch.zeros(800, dtype=torch.bool)
    hit[[7, 401, 500]] = True
    assert not torch.isfinite(y[hit]).any()
    hit[600] = True
    v, e = R.linear(x, w, off)
    R.assert_close(y[~hit], v[~hit], e[~hit])


# ---------------------------------------------------------------- 8-bit rows


def special_rows(k):
    """Rows around every decision of the format: scale borders, ties, tiny and
    huge magnitudes, signed zeros, infinities and NaN."""
    v = R.normal(11, 24, k, dtype=F32)
    v *= torch.exp2(torch.linspace(-150, 120, 24))[:, None]
    v[0] = 0.0
    v[1] = -0.0
    v[2, 0] = 448.0
    v[3] = v[3].clamp(-440, 440)
    v[3, 0] = 448.0 * (1 + 2.0 ** -7)
    v[4, -1] = float("inf")
    v[5, 0] = float("-inf")
    v[6, k // 2] = float("nan")
    v[7] = float("nan")
    v[8, 0] = 3.3e38
    v[9] = torch.arange(k) % 17 - 8.0
    v[10] = 2.0 ** -149
    return v


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [1, 31, 32, 33, 40, 64, 256, 1000, 4104])
def test_checkpoint_rows(k, dtype):
    v = torch.cat([special_rows(k), R.normal(12, 100, k, dtype=F32)]).to(dtype)
    c = moe.checkpoint_rows(v.cuda())
    exps = R.scale_exps(v)
    codes, bad = R.e4m3_codes(v, exps)
    assert torch.equal(c.exps.cpu(), exps)
    got = c.codes.cpu()
    assert ((got & 0x7F)[bad] == 0x7F).all()
    assert torch.equal(got[~bad], codes[~bad])
    # read back: in order, and gathered with rows repeated, in both types
    idx = torch.randint(len(v), (211,), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    idx[:3] = 7
    want = R.decode(got, exps)
    for out in (BF, F32):
        for index, w in ((None, want), (idx.cuda(), want[idx.long()])):
            r = moe.restore_rows(c, index, dtype=out).cpu()
            assert r.dtype == out
            assert torch.equal(torch.isnan(r), torch.isnan(w))
            f = ~torch.isnan(w)
            assert torch.equal(r[f], w[f].to(out))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [255, 256])
def test_every_code_with_every_scale(k, dtype):
    # row e holds the codes under the scale byte e; NaN codes make their blocks
    # take another way, so the rows come without them too
    codes = torch.arange(256, dtype=torch.int16).repeat(256, 1)[:, :k]
    finite = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes)
    codes = torch.cat([codes, finite]).to(torch.uint8).contiguous()
    exps = torch.arange(256).to(torch.uint8).repeat(2)[:, None].repeat(1, (k + 31) // 32).contiguous()
    got = moe.restore_rows(moe.Checkpoint(codes.cuda(), exps.cuda()), dtype=dtype).cpu()
    # 2^(byte - 127) in 64 bits; byte 255 reads as an infinity, which makes zeros NaN
    scale = torch.ldexp(torch.ones(512, 1, dtype=torch.float64), exps[:, :1].int() - 127)
    scale[exps[:, :1] == 255] = float("inf")
    want = (codes.view(torch.float8_e4m3fn).double() * scale).to(torch.float32).to(dtype)
    assert torch.equal(got.isnan(), want.isnan())
    ok = ~want.isnan()
    assert torch.equal(got[ok], want[ok])
    assert torch.equal(got[ok].signbit(), want[ok].signbit())


def test_restore_rows_refuses_bad_indices():
    v = R.normal(1, 10, 96)
    c = moe.checkpoint_rows(v.cuda())
    for k in (96, 33):
        c = moe.checkpoint_rows(v[:, :k].contiguous().cuda())
        st = status()
        idx = torch.tensor([0, -1, 9, 10, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
        r = moe.restore_rows(c, idx, status=st)
        assert int(st.item()) == -6
        assert (r[[1, 3, 4, 5]] == 0).all()
        assert torch.equal(r[[0, 2]], moe.restore_rows(c)[[0, 9]])


# ------------------------------------------------- SwiGLU with its checkpoint


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes,n,k", SHAPES)
def test_swiglu_checkpoint(sizes, n, k, dtype):
    off = R.offsets_of(sizes)
    rows, G = off[-1], len(sizes)
    x = R.normal(1, rows, k, dtype=dtype)
    w1, w3 = (R.normal(i, G, n, k, dtype=dtype, std=2 * k ** -0.5) for i in (2, 3))
    st = status()
    h, a, u = moe.swiglu_checkpoint(*dev(x, w1, w3), offs(off), status=st)
    assert int(st.item()) == 0
    (av, ae), (uv, ue) = R.linear(x, w1, off), R.linear(x, w3, off)
    # |silu'| <= 1.1
    s = R.silu(av).abs()
    err = 1.1 * ae * (uv.abs() + ue) + s * ue + s * uv.abs() * (R.sigmoid_rel(av, dtype) + 4 * R.ULP)
    R.assert_close(h, R.silu(av) * uv, err, "h")
    for c, v, e in ((a, av, ae), (u, uv, ue)):
        exps = c.exps.cpu()
        # the scale is the definition's for some value within the sum's error
        nb = exps.shape[1]
        pad = torch.nn.functional.pad(torch.stack([v.abs() - e, v.abs() + e]), (0, 32 * nb - n))
        low, high = pad.reshape(2, rows, nb, 32).amax(3)
        assert (low <= 448 * torch.exp2(exps.to(R.F64) - 127)).all()
        assert ((high > 224 * torch.exp2(exps.to(R.F64) - 127)) | (exps == 0)).all()
        # a code is off by half a step: 2^-4 of the value, or 2^-10 of the scale
        scale = torch.exp2(exps.to(R.F64) - 127).repeat_interleave(32, 1)[:, :n]
        d = (R.decode(c.codes.cpu(), exps) - v).abs()
        assert (d <= torch.maximum(2.0 ** -4 * (v.abs() + e), scale * 2.0 ** -10) + e).all()


def backward_case(sizes, n, k, dtype, first=0, spare=0):
    off = R.offsets_of(sizes, first)
    rows, G = off[-1] + spare, len(sizes)
    dy = R.normal(1, rows, k, dtype=dtype)
    w2 = R.normal(2, G, k, n, dtype=dtype, std=n ** -0.5)
    a, u = (moe.checkpoint_rows(R.normal(i, rows, n, dtype=F32, std=2.0).cuda()) for i in (3, 4))
    gate = torch.rand(rows, generator=torch.Generator().manual_seed(5)) + 0.1
    return off, dy, w2, a, u, gate


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("sizes,n,k", SHAPES)
def test_swiglu_backward(sizes, n, k, gated, dtype):
    off, dy, w2, a, u, gate = backward_case(sizes, n, k, dtype)
    if not gated:
        gate = torch.ones_like(gate)
    st = status()
    got = moe.swiglu_backward(*dev(dy, w2), a, u, offs(off), gate=gate.cuda() if gated else None,
                              status=st)
    assert int(st.item()) == 0
    dh, e = R.dx(dy, w2, off)
    av, uv = (R.decode(c.codes.cpu(), c.exps.cpu()) for c in (a, u))
    vals, errs = R.swiglu_grads(av, uv, dh, e, gate.to(R.F64), dtype)
    for g, v, b, name in zip(got, vals, errs, ("da", "du", "hg", "dgate")):
        R.assert_close(g, v, b, name)


def test_swiglu_backward_against_differences():
    """The formulas above are the derivatives of gate * (silu(a) u) w2^T . dy:
    central differences in 64 bits, and the kernel's against them."""
    off, dy, w2, a, u, gate = backward_case([3, 0, 5], 40, 24, F32)
    av, uv = (R.decode(c.codes.cpu(), c.exps.cpu()) for c in (a, u))
    gd, dyd = gate.to(R.F64), dy.to(R.F64)

    def loss(av, uv, gd):
        h = R.silu(av) * uv
        return (gd[:, None] * R.linear(h, w2.transpose(1, 2).to(R.F64).transpose(1, 2), off)[0] * dyd).sum(1)

    da, du, hg, dgate = (t.cpu().to(R.F64) for t in moe.swiglu_backward(
        *dev(dy, w2), a, u, offs(off), gate=gate.cuda()))
    eps = 1e-5
    for i in range(0, 40, 7):
        step = torch.zeros_like(av)
        step[:, i] = eps
        for got, lo, hi in ((da, loss(av - step, uv, gd), loss(av + step, uv, gd)),
                            (du, loss(av, uv - step, gd), loss(av, uv + step, gd))):
            # fp32 results of a few units: 1e-4 covers their 2^-23 * 24 terms,
            # and the differences' eps^2
            assert ((hi - lo) / (2 * eps) - got[:, i]).abs().max() < 1e-4
    assert ((loss(av, uv, gd + eps) - loss(av, uv, gd - eps)) / (2 * eps) - dgate).abs().max() < 2e-4


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,k", [(128, 256), (200, 264), (33, 77)])
def test_swiglu_rows_outside_the_groups_stay(n, k, dtype):
    off, dy, w2, a, u, gate = backward_case([33, 0, 4], n, k, dtype, first=2, spare=20)
    nan = float("nan")
    dy[:2] = nan
    dy[off[-1]:] = nan
    gate[off[-1]:] = nan
    rows = dy.shape[0]
    live = slice(off[0], off[-1])
    from sparse_moe_layer_sum_b200 import training
    marks = {}
    empty = torch.empty

    def marked(*shape, **kw):
        t = empty(*shape, **kw)
        t.view(-1).view(torch.uint8).fill_(0x3B) if t.numel() else None
        marks[t.data_ptr()] = t
        return t

    training.torch.empty = marked
    try:
        got = moe.swiglu_backward(*dev(dy, w2), a, u, offs(off), gate=gate.cuda())
        x = R.normal(9, rows, k, dtype=dtype)
        x[:2] = nan
        w1 = R.normal(8, 3, n, k, dtype=dtype)
        h, ca, cu = moe.swiglu_checkpoint(*dev(x, w1, w1), offs(off))
    finally:
        training.torch.empty = empty
    for t in (*got, h, ca.codes, ca.exps, cu.codes, cu.exps):
        b = t.contiguous().view(rows, -1).view(torch.uint8).cpu()
        assert (b[:2] == 0x3B).all() and (b[off[-1]:] == 0x3B).all()
        if t.dtype != torch.uint8:
            assert torch.isfinite(t[live]).all()


# ------------------------------------------------------------- how it is called


def test_bad_offsets_are_clamped_and_reported():
    x, w = R.normal(1, 40, 64).cuda(), R.normal(2, 3, 64, 64).cuda()
    dy = R.normal(3, 40, 64).cuda()
    a = moe.checkpoint_rows(R.normal(4, 40, 64).cuda())
    for off in ([0, 20, 10, 40], [0, 10, 20, 41], [-5, 10, 20, 40], [0, 2 ** 31 - 1, 20, 40],
                [50, 60, 70, 80]):
        for call in (lambda o, s: moe.grouped_linear(x, w, o, status=s),
                     lambda o, s: moe.grouped_linear_dx(dy, w, o, status=s),
                     lambda o, s: moe.grouped_linear_dw(dy, x, o, status=s),
                     lambda o, s: moe.swiglu_checkpoint(x, w, w, o, status=s),
                     lambda o, s: moe.swiglu_backward(dy, w, a, a, o, status=s)):
            st = status()
            call(offs(off), st)
            assert int(st.item()) == -6, off


def test_no_rows():
    o = offs([0, 0, 0])
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), R.normal(1, 2, 72, 64).cuda()
    dy = torch.empty(0, 72, dtype=BF, device="cuda")
    assert moe.grouped_linear(x, w, o).shape == (0, 72)
    assert moe.grouped_linear_dx(dy, w, o).shape == (0, 64)
    dw = moe.grouped_linear_dw(dy, x, o)
    assert dw.shape == (2, 72, 64) and (dw == 0).all()
    h, a, u = moe.swiglu_checkpoint(x, w, w, o)
    assert h.shape == (0, 72) and a.codes.shape == (0, 72) and u.exps.shape == (0, 3)
    w2 = R.normal(2, 2, 64, 72).cuda()
    assert [t.shape for t in moe.swiglu_backward(x, w2, a, u, o)] == [(0, 72)] * 3 + [(0,)]
    c = moe.checkpoint_rows(x)
    assert moe.restore_rows(c).shape == (0, 64)


def test_rows_that_belong_to_no_group():
    """Rows, but only empty groups: nothing is written, and dw is zero."""
    x, w = R.normal(1, 64, 128).cuda(), R.normal(2, 3, 96, 128).cuda()
    y = torch.full((64, 96), 5.0, dtype=BF, device="cuda")
    for at in (0, 7, 64):
        o = offs([at] * 4)
        assert moe.grouped_linear(x, w, o, out=y) is y and (y == 5).all()
        assert (moe.grouped_linear_dw(y, x, o) == 0).all()
        base = R.normal(3, 3, 96, 128, dtype=F32).cuda()
        acc = base.clone()
        moe.grouped_linear_dw(y, x, o, out=acc, accumulate=True)
        assert torch.equal(acc, base)
        h, a, u = moe.swiglu_checkpoint(x, w, w, o)
        moe.swiglu_backward(x, w.transpose(1, 2).contiguous(), a, u, o)


def test_calls_from_several_threads():
    import threading
    t = chain_inputs(60)
    want = run_all(t)
    torch.cuda.synchronize()
    same = {}

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = run_all(t)
            s.synchronize()
            same[i] = all(torch.equal(a, b) for a, b in zip(got, want))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert same == {0: True, 1: True, 2: True}


def run_all(t):
    """Every operator once, chained as a backward pass would; results in a list."""
    h, a, u = moe.swiglu_checkpoint(t["x"], t["w1"], t["w3"], t["off"])
    y = moe.grouped_linear(h, t["w2"], t["off"])
    da, du, hg, dgate = moe.swiglu_backward(t["dy"], t["w2"], a, u, t["off"], gate=t["gate"])
    dx = moe.grouped_linear_dx(da, t["w1"], t["off"], dy2=du, w2=t["w3"])
    xr = moe.restore_rows(moe.checkpoint_rows(t["x"]), t["index"])
    return [h, y, da, du, hg, dgate, dx, xr, moe.grouped_linear_dw(da, xr, t["off"]),
            moe.grouped_linear_dw(t["dy"], hg, t["off"], out_dtype=F32)]


def chain_inputs(seed, sizes=(70, 0, 131, 5), n=256, k=384):
    off = R.offsets_of(sizes)
    G, rows = len(sizes), off[-1]
    t = dict(x=R.normal(seed, rows, k), dy=R.normal(seed + 1, rows, k),
             w1=R.normal(seed + 2, G, n, k, std=k ** -0.5), w3=R.normal(seed + 3, G, n, k, std=k ** -0.5),
             w2=R.normal(seed + 4, G, k, n, std=n ** -0.5))
    t = {a: b.cuda() for a, b in t.items()}
    t["gate"] = torch.rand(rows, generator=torch.Generator().manual_seed(seed)).cuda()
    t["off"] = offs(off)
    t["index"] = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda")
    return t


@pytest.mark.parametrize("n,k", [(256, 384), (100, 77)])
def test_repeatable_on_streams_and_in_graphs(n, k):
    t = chain_inputs(20, n=n, k=k)
    want = run_all(t)
    for a, b in zip(want, run_all(t)):
        assert torch.equal(a, b)
    # two streams at once, other inputs on the second
    t2 = chain_inputs(40, n=n, k=k)
    want2 = run_all(t2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        r1 = [run_all(t) for _ in range(3)][-1]
    with torch.cuda.stream(s2):
        r2 = [run_all(t2) for _ in range(3)][-1]
    torch.cuda.synchronize()
    for w, r in ((want, r1), (want2, r2)):
        assert all(torch.equal(a, b) for a, b in zip(w, r))
    # two captured graphs, replayed in turn on inputs changed in place
    graphs = []
    for src in (t, t2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run_all(src)
        graphs.append((g, out))
    for (g, out), w in zip(graphs * 2, (want, want2) * 2):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    t["off"].copy_(offs([0, 1, 100, 206, 206]))
    g, out = graphs[0]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, run_all(t)))


def test_refusals():
    x, w, o = R.normal(1, 8, 64).cuda(), R.normal(2, 2, 32, 64).cuda(), offs([0, 4, 8])
    bad = [
        lambda: moe.grouped_linear(x.cpu(), w, o),
        lambda: moe.grouped_linear(x.t(), w, o),
        lambda: moe.grouped_linear(x[:, :32], w, o),
        lambda: moe.grouped_linear(x.half(), w.half(), o),
        lambda: moe.grouped_linear(x.float(), w, o),
        lambda: moe.grouped_linear(x, w, o.long()),
        lambda: moe.grouped_linear(x, w, o[:2]),
        lambda: moe.grouped_linear(x, w, o, out=torch.empty(8, 31, dtype=BF, device="cuda")),
        lambda: moe.grouped_linear(x, w, o, out_dtype=torch.float16),
        lambda: moe.grouped_linear_dx(x, w, o),
        lambda: moe.grouped_linear_dx(x[:, :32].contiguous(), w, o, dy2=x[:, :32].contiguous()),
        lambda: moe.grouped_linear_dw(x, x[:4], o),
        lambda: moe.grouped_linear_dw(x, x, o, accumulate=True),
        lambda: moe.checkpoint_rows(x[0]),
        lambda: moe.restore_rows(moe.checkpoint_rows(x), o.long()),
        lambda: moe.restore_rows(moe.Checkpoint(x.view(torch.uint8), x.view(torch.uint8))),
        lambda: moe.swiglu_checkpoint(x, w, w[:1], o),
        lambda: moe.swiglu_backward(x, w.transpose(1, 2).contiguous(), moe.checkpoint_rows(x),
                                    moe.checkpoint_rows(x), o),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was accepted")
