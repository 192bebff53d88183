"""Calls of the training binding that are refused before anything reaches the
GPU, so that they are tested without one."""
import pytest
import torch

import sparse_moe_layer_sum_b200 as moe

SHAPE = moe.BlockShape(dim=64, n_routed=8, n_groups=2, topk_groups=1, topk=2, inter=32, n_shared=0)
SHARED = moe.BlockShape(dim=64, n_routed=8, n_groups=2, topk_groups=1, topk=2, inter=32, n_shared=1)


def params(shape):
    G = shape.n_routed + shape.n_shared
    w = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    return moe.BlockParams(torch.zeros(shape.n_routed, shape.dim), None, w(G, shape.inter, shape.dim),
                           w(G, shape.inter, shape.dim), w(G, shape.dim, shape.inter))


def routing(shape, T):
    i32 = torch.int32
    return (torch.zeros(T, shape.topk), torch.zeros(shape.n_routed + 1, dtype=i32),
            torch.zeros(T * shape.topk, dtype=i32), torch.zeros(T * shape.topk, dtype=i32))


def saved(shape, T, slots=None, rows=None):
    u8, i32 = torch.uint8, torch.int32
    R = T * (shape.topk + shape.n_shared) if rows is None else rows
    ckpt = lambda n, k: moe.Checkpoint(torch.zeros(n, k, dtype=u8), torch.zeros(n, -(-k // 32), dtype=u8))
    return moe.SavedExperts(ckpt(T, shape.dim), ckpt(R, shape.inter), ckpt(R, shape.inter),
                            torch.zeros(R, dtype=i32), torch.zeros(R),
                            torch.zeros(shape.n_routed + shape.n_shared + 1, dtype=i32),
                            torch.zeros(T * shape.topk if slots is None else slots, dtype=i32),
                            torch.bfloat16)


@pytest.mark.parametrize("shape", [SHAPE, SHARED], ids=["routed", "shared"])
@pytest.mark.parametrize("T", [7, 9, 16])
def test_forward_takes_the_routing_of_its_own_rows(shape, T):
    """x of more or fewer tokens than the routing was made for."""
    x = torch.zeros(T, shape.dim, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="routing"):
        moe.experts_training_forward(shape, params(shape), x, *routing(shape, 8))
    # the weights of T tokens with the lists of 8
    with pytest.raises(ValueError, match="routing"):
        moe.experts_training_forward(shape, params(shape), x, torch.zeros(T, shape.topk),
                                     *routing(shape, 8)[1:])


@pytest.mark.parametrize("shape", [SHAPE, SHARED], ids=["routed", "shared"])
def test_backward_takes_lists_of_the_saved_batch(shape):
    dy = torch.zeros(16, shape.dim)
    p = params(shape)
    R = 8 * (shape.topk + shape.n_shared)
    for s in (saved(shape, 16, slots=8 * shape.topk), saved(shape, 16, rows=R),
              saved(shape, 16, slots=8 * shape.topk, rows=R),
              saved(SHAPE if shape is SHARED else SHARED, 16)):
        with pytest.raises(ValueError, match="saved"):
            moe.experts_training_backward(shape, p, s, dy)


@pytest.mark.parametrize("name", ["dw1", "dw3", "dw2"])
def test_no_gradient_is_added_to_when_one_does_not_fit(name):
    p = params(SHAPE)
    good = dict(dx=None, dgates=None, dw1=torch.zeros_like(p.w1), dw3=torch.zeros_like(p.w3),
                dw2=torch.zeros_like(p.w2))
    with pytest.raises(ValueError, match="CUDA"):         # fits
        moe.experts_training_backward(SHAPE, p, saved(SHAPE, 16), torch.zeros(16, SHAPE.dim),
                                      accumulate=moe.ExpertGrads(**good))
    for bad in (good[name][:-1], good[name].double(), good[name].transpose(1, 2)):
        with pytest.raises(ValueError, match="accumulate"):
            moe.experts_training_backward(SHAPE, p, saved(SHAPE, 16), torch.zeros(16, SHAPE.dim),
                                          accumulate=moe.ExpertGrads(**{**good, name: bad}))


@pytest.mark.parametrize("shape", [SHAPE, SHARED], ids=["routed", "shared"])
def test_combine_reads_within_its_operands(shape):
    T, n = 8, 8 * shape.topk
    good = dict(weights=torch.zeros(T, shape.topk), slot_of=torch.zeros(n, dtype=torch.int32),
                out_perm=torch.zeros(n, shape.dim),
                out_shared=torch.zeros(T, shape.dim) if shape.n_shared else None)
    with pytest.raises(ValueError, match="CUDA"):
        moe.combine(shape, **good)
    bad = dict(weights=torch.zeros(T, 1), slot_of=good["slot_of"][:-1], out_perm=good["out_perm"][:-1],
               y=torch.zeros(T - 1, shape.dim))
    if shape.n_shared:
        bad["out_shared"] = good["out_shared"][:-1]
    for name, v in bad.items():
        with pytest.raises(ValueError, match="one batch"):
            moe.combine(shape, **{**good, name: v})
    if shape.n_shared:
        with pytest.raises(ValueError, match="one batch"):
            moe.combine(shape, **{**good, "out_shared": None})
    for name, v in (("out_perm", good["out_perm"].bfloat16()), ("slot_of", good["slot_of"].short()),
                    ("y", torch.zeros(T, shape.dim, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="fp32"):
            moe.combine(shape, **{**good, name: v})


def test_training_rows_of_a_wrapping_token_count():
    """T * (topk + n_shared) past 64 bits: 2^61 * 8 is 0 there."""
    import ctypes
    from sparse_moe_layer_sum_b200 import build
    from sparse_moe_layer_sum_b200._lib import MoECfg, fn
    build.build_all()
    p = ctypes.c_void_p(0x1000)                     # never dereferenced
    cfg = MoECfg(dim=64, n_routed=8, n_groups=1, topk_groups=1, topk=7, inter=32, n_shared=1,
                 route_scale=2.5, score_func=0, has_bias=1)
    for T in (1 << 61, 1 << 62, (1 << 61) + 1):
        assert fn("moe_train", "moe_training_rows")(ctypes.byref(cfg), T, p, p, p, p, p, p, p, None,
                                                    None) == -2


def test_workspace_for_any_operands_is_enough_for_aligned_ones():
    import ctypes
    import random
    from sparse_moe_layer_sum_b200 import build
    from sparse_moe_layer_sum_b200._lib import MoEGroupedShape, fn
    build.build_all()
    rng = random.Random(3)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    shapes = [(16, 300, 1024, 16), (1, 816, 168, 1710)]      # parts of a tensor-core product
    shapes += [(log(1, 300), log(1, 8192), log(1, 8192), log(1, 70000)) for _ in range(3000)]
    more = 0
    for shape in shapes:
        s = ctypes.byref(MoEGroupedShape(*shape))
        for dt in (0, 1):
            for name, flags in (("grouped_linear", ()), ("grouped_linear_dx", (0,)), ("grouped_linear_dx", (1,)),
                                ("grouped_linear_dw", ()), ("swiglu_checkpoint", ()), ("swiglu_backward", ())):
                size = fn("moe_train", f"moe_{name}_workspace_size")
                one, any_ = size(s, dt, *flags, 1), size(s, dt, *flags, 0)
                assert any_ >= one, (name, shape, dt)
                more += any_ > one
    assert more > 0


def test_out_apart_from_the_operands():
    from sparse_moe_layer_sum_b200.training import _apart
    buf = torch.zeros(256)
    x = buf[64:128]
    for lo, hi in ((64, 128), (0, 65), (127, 200), (0, 256), (80, 81)):
        with pytest.raises(ValueError, match="share memory"):
            _apart(buf[lo:hi], (None, torch.zeros(3), x))
    for lo, hi in ((0, 64), (128, 256), (70, 70)):
        _apart(buf[lo:hi], (None, x))
    _apart(buf[64:128], (x[:0],))
