"""The experts' forward and backward pass on the block's own routing, against
64-bit autograd on the CPU, element by element.

The backward pass uses the batch and the projections as the checkpoint holds
them, so the reference's graph does too: each is replaced by its decoded value
with the gradient passed through.  What is left between the two are the fp32
sums and the roundings to the operand type, whose bounds are carried along
(train_ref)."""
from dataclasses import replace

import pytest
import torch

import train_ref as R
import sparse_moe_layer_sum_b200 as moe
from sparse_moe_layer_sum_b200.inputs import custom, make_block

pytestmark = pytest.mark.gpu

F64, F32, BF = torch.float64, torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_moe_layer_sum_b200 import build
    build.build_all()


def setup(T, dtype, n_shared=1, **kw):
    sh = dict(dim=256, n_routed=16, n_groups=4, topk_groups=2, topk=4, inter=128)
    sh.update(kw)
    w = custom("train", T, x_dtype=dtype, w_format="bf16" if dtype == BF else "f32", seed=31,
               n_shared=n_shared, **sh)
    x, p = make_block(w, "cuda:0")
    weights, indices, _ = moe.router_forward(w.shape, x, p.w_r, p.bias)
    _, offsets, sorted_token, slot_of = moe.dispatch_build(w.shape, indices)
    return w.shape, x, p, weights, (offsets, sorted_token, slot_of)


def autograd(t, dec, w1, w3, w2, off, token, gate, T):
    """y and the gradients for dy, with t, a, u at their decoded values."""
    for v in (t["x"], w1, w3, w2, gate):
        v.requires_grad_()
    x = t["x"] + (dec["x"] - t["x"]).detach()
    y = torch.zeros(T, t["x"].shape[1], dtype=F64)
    for g, r in R.groups(off):
        if r.stop == r.start:
            continue
        rows = x[token[r]]
        a, u = rows @ w1[g].T, rows @ w3[g].T
        a = a + (dec["a"][r] - a).detach()
        u = u + (dec["u"][r] - u).detach()
        o = (R.silu(a) * u) @ w2[g].T
        y = y.index_add(0, token[r], gate[r, None] * o)
    (y * t["dy"]).sum().backward()
    return t["x"].grad, gate.grad, w1.grad, w3.grad, w2.grad


CASES = [
    dict(T=64, dtype=BF), dict(T=64, dtype=F32),
    dict(T=1, dtype=BF), dict(T=33, dtype=BF, n_shared=0),
    dict(T=300, dtype=BF, dim=512, inter=320, n_routed=4, n_groups=1, topk_groups=1, topk=2),
    dict(T=50, dtype=BF, dim=200, inter=72), dict(T=50, dtype=F32, dim=100, inter=77),
    dict(T=40, dtype=BF, dim=100, inter=77),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_forward_and_backward(case):
    shape, x, p, weights, (offsets, sorted_token, slot_of) = setup(**case)
    T, k, dtype = case["T"], shape.topk, case["dtype"]
    half = R.HALF[dtype]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, saved = moe.experts_training_forward(shape, p, x, weights, offsets, sorted_token, slot_of, status=st)
    dy = R.normal(77, T, shape.dim, dtype=F32).cuda()
    grads = moe.experts_training_backward(shape, p, saved, dy, status=st)
    assert int(st.item()) == 0

    # the row lists, from the routing alone
    S, E = shape.n_shared, shape.n_routed
    slots = slot_of.cpu().long().view(T, k)
    token = torch.cat([sorted_token.cpu().long(), torch.arange(T)[:T * S]])
    gate = torch.ones(T * (k + S))
    gate[slots.view(-1)] = weights.cpu().view(-1)
    off = offsets.cpu().tolist() + ([T * (k + 1)] if S else [])
    assert torch.equal(saved.row_token.cpu().long(), token)
    assert torch.equal(saved.row_gate.cpu(), gate)
    assert saved.group_offsets.cpu().tolist() == off

    w1, w3, w2 = (t.cpu() for t in (p.w1, p.w3, p.w2))
    gd = gate.to(F64)[:, None]

    def tokens(rows):  # sums of the rows of each token
        return torch.zeros(T, rows.shape[1], dtype=F64).index_add(0, token, rows)

    # forward
    xr = x.cpu()[token]
    (a, ae), (u, ue) = R.linear(xr, w1, off), R.linear(xr, w3, off)
    s = R.silu(a).abs()
    h = R.silu(a) * u
    he = 1.1 * ae * (u.abs() + ue) + s * ue + h.abs() * (R.sigmoid_rel(a, dtype) + 4 * R.ULP)
    he = he + half * (h.abs() + he)
    o, _ = R.linear(h, w2, off)
    mag = R.linear(h.abs() + he, w2.abs(), off)[0]
    oe = R.linear(he, w2.abs(), off)[0] + (shape.inter + 1) * R.ULP * mag
    R.assert_close(y, tokens(gd * o), tokens(gd * (oe + (k + 2) * R.ULP * (o.abs() + oe))), "y")

    # backward
    dec = {n: R.decode(c.codes.cpu(), c.exps.cpu()) for n, c in (("x", saved.x), ("a", saved.a), ("u", saved.u))}
    dyr = dy.cpu().to(dtype)
    t = dict(x=x.cpu().to(F64), dy=dyr.to(F64))
    W = [m.to(F64) for m in (w1, w3, w2)]
    ref = autograd(t, dec, *W, off, token, gate.to(F64), T)
    dx, dgate, dw1, dw3, dw2 = ref

    W = [m.detach() for m in W]
    dh, e = R.dx(dyr[token], w2, off)
    (da, du, hg, _), (eda, edu, ehg, edg) = R.swiglu_grads(dec["a"], dec["u"], dh, e, gate.to(F64), dtype)
    eda, edu, ehg = (b + half * (v.abs() + b) for v, b in ((da, eda), (du, edu), (hg, ehg)))
    xs = dec["x"][token]
    for got, want, d, ed, rows in ((grads.dw1, dw1, da, eda, xs), (grads.dw3, dw3, du, edu, xs),):
        err = R.dw(d.abs() + ed, rows, off)[1] + R.dw(ed, rows.abs(), off)[0]
        R.assert_close(got, want, err, "dw1 dw3")
    err = R.dw(dyr[token], hg.abs() + ehg, off)[1] + R.dw(dyr[token].to(F64).abs(), ehg, off)[0]
    R.assert_close(grads.dw2, dw2, err, "dw2")
    rows, re = R.dx(da.abs() + eda, W[0].abs(), off, du.abs() + edu, W[1].abs())
    re = re + R.dx(eda, W[0].abs(), off, edu, W[1].abs())[0]
    R.assert_close(grads.dx, dx, tokens(re + (k + 2) * R.ULP * rows), "dx")
    R.assert_close(grads.dgates, dgate[slots], edg[slots], "dgates")


def test_gradients_accumulate_and_repeat():
    shape, x, p, weights, route = setup(64, BF)
    dy = R.normal(5, 64, shape.dim, dtype=F32).cuda()
    y, saved = moe.experts_training_forward(shape, p, x, weights, *route)
    y2, _ = moe.experts_training_forward(shape, p, x, weights, *route)
    assert torch.equal(y, y2)                                 # no atomics
    g = moe.experts_training_backward(shape, p, saved, dy)
    g2 = moe.experts_training_backward(shape, p, saved, dy)
    for n in ("dx", "dgates", "dw1", "dw3", "dw2"):
        assert torch.equal(getattr(g, n), getattr(g2, n)), n
    once = replace(g, dw1=g.dw1.clone(), dw3=g.dw3.clone(), dw2=g.dw2.clone())
    acc = moe.experts_training_backward(shape, p, saved, dy, accumulate=g2)
    for n in ("dw1", "dw3", "dw2"):
        assert getattr(acc, n) is getattr(g2, n)
        assert torch.equal(getattr(acc, n), 2 * getattr(once, n)), n   # v + v is exact
    half = moe.experts_training_backward(shape, p, saved, dy, grad_dtype=BF)
    assert torch.equal(half.dw1, once.dw1.to(BF))
    # the checkpoint is about half of the bf16 activations it stands for
    R_ = 64 * (shape.topk + 1)
    full = 2 * (64 * shape.dim + 2 * R_ * shape.inter)
    assert saved.nbytes < 0.52 * full


def test_empty_batch_and_refusals():
    shape, x, p, weights, route = setup(4, BF)
    e = x[:0]
    w0, i0, _ = moe.router_forward(shape, x, p.w_r, p.bias)
    _, o0, s0, l0 = moe.dispatch_build(shape, i0[:0])
    y, saved = moe.experts_training_forward(shape, p, e, w0[:0], o0, s0, l0)
    g = moe.experts_training_backward(shape, p, saved, e)
    assert y.shape == (0, shape.dim) and g.dx.shape == (0, shape.dim) and g.dgates.shape == (0, shape.topk)
    assert (g.dw1 == 0).all() and (g.dw2 == 0).all()
    y, saved = moe.experts_training_forward(shape, p, x, weights, *route)
    with pytest.raises(ValueError):
        moe.experts_training_backward(shape, p, saved, x[:2])
    with pytest.raises(ValueError):
        moe.experts_training_forward(shape, p, x.float(), weights, *route)
    with pytest.raises(ValueError):
        moe.experts_training_forward(shape, p, x, weights[:, :2].contiguous(), *route)
    with pytest.raises(ValueError):
        moe.gather_rows(x, route[2].long())


def test_gather_rows_and_bad_indices():
    for k in (64, 40, 33, 1):
        for dt in (BF, F32):
            v = R.normal(3, 9, k, dtype=dt)
            idx = torch.tensor([8, 0, 0, 3, -1, 9], dtype=torch.int32, device="cuda")
            for out in (BF, F32):
                st = torch.zeros(1, dtype=torch.int32, device="cuda")
                got = moe.gather_rows(v.cuda(), idx, dtype=out, status=st).cpu()
                assert int(st.item()) == -6
                assert torch.equal(got[:4], v[[8, 0, 0, 3]].to(out)) and (got[4:] == 0).all()


def test_bad_slots_are_reported():
    shape, x, p, weights, (offsets, sorted_token, slot_of) = setup(16, BF)
    for tok, slot in ((-1, 0), (16, 0), (0, -1), (0, 16 * shape.topk)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        a, b = sorted_token.clone(), slot_of.clone()
        a[3], b[5] = tok, slot
        moe.training_rows(shape, weights, offsets, a, b, status=st)
        assert int(st.item()) == -6


def test_captured_step():
    """A whole step in one graph, replayed on other batches: the routing, and
    with it every group's length, changes between the replays."""
    shape, x, p, _, _ = setup(64, BF)
    dy = R.normal(5, 64, shape.dim, dtype=F32).cuda()

    def step():
        w, idx, _ = moe.router_forward(shape, x, p.w_r, p.bias)
        _, *route = moe.dispatch_build(shape, idx)
        y, saved = moe.experts_training_forward(shape, p, x, w, *route)
        g = moe.experts_training_backward(shape, p, saved, dy)
        return [y, g.dx, g.dgates, g.dw1, g.dw3, g.dw2]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2):
        x.copy_(R.normal(seed, 64, shape.dim).cuda())
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))
