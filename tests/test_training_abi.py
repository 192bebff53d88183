"""moe_train without a GPU: what it exports, and what it refuses before any
CUDA call."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from conftest import ROOT
import train_ref as R
from sparse_moe_layer_sum_b200 import _lib
from sparse_moe_layer_sum_b200._lib import MoEGroupedShape, fn

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = ctypes.c_void_p(0x1000)  # a non-null pointer that is never dereferenced
F32, BF16, E4M3 = 0, 1, 2


@pytest.fixture(scope="module", autouse=True)
def built():
    from sparse_moe_layer_sum_b200 import build
    build.build_all()


def shape(groups=4, n=64, k=128, rows=10):
    return ctypes.byref(MoEGroupedShape(groups, n, k, rows))


def test_exports_are_the_header():
    text = open(os.path.join(ROOT, "include", "moe_train.h")).read()
    names = re.findall(r"^(?:moe_status|size_t)\s+(\w+)\s*\(", text, flags=re.M)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.lib_path("moe_train")],
                         capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert {e for e in exported if e.startswith("moe_")} == set(names)
    assert {s for lib, s in _lib.SIGNATURES if lib == "moe_train"} == set(names)


BAD_SHAPES = [(dict(groups=0), INVALID), (dict(n=0), INVALID), (dict(k=-1), INVALID),
              (dict(rows=-1), INVALID), (dict(groups=1025), UNSUPPORTED),
              (dict(rows=1 << 31), UNSUPPORTED), (dict(n=(1 << 20) + 1), UNSUPPORTED),
              (dict(n=1 << 20, rows=(1 << 31) - 1), UNSUPPORTED)]


def linear(s, x=P, dt=BF16, w=P, off=P, y=P, ydt=BF16):
    return fn("moe_train", "moe_grouped_linear")(s, x, dt, w, off, y, ydt, None, 0, None, None)


def dx(s, dy=P, dt=BF16, w=P, dy2=None, w2=None, off=P, out=P, odt=BF16):
    return fn("moe_train", "moe_grouped_linear_dx")(s, dy, dt, w, dy2, w2, off, out, odt, None, 0, None,
                                                  None)


def dw(s, dy=P, dt=BF16, x=P, off=P, out=P, odt=BF16, acc=0):
    return fn("moe_train", "moe_grouped_linear_dw")(s, dy, dt, x, off, out, odt, acc, None, 0, None, None)


def save(s, x=P, dt=BF16, h=P, ca=P, ws=P, nws=1 << 40):
    return fn("moe_train", "moe_swiglu_checkpoint")(s, x, dt, P, P, P, h, ca, P, P, P, ws, nws, None,
                                                    None)


def back(s, dy=P, dt=BF16, ca=P, dgate=P, ws=P, nws=1 << 40):
    return fn("moe_train", "moe_swiglu_backward")(s, dy, dt, P, ca, P, P, P, None, P, P, P, P, dgate,
                                                  ws, nws, None, None)


@pytest.mark.parametrize("call", [linear, dx, dw, save, back])
def test_shapes_and_types(call):
    for kw, want in BAD_SHAPES:
        assert call(shape(**kw)) == want, kw
    assert call(None) == INVALID
    for dt in (E4M3, 7, -1):
        assert call(shape(), dt=dt) == UNSUPPORTED


def test_missing_pointers():
    for call, names in ((linear, ("x", "w", "off", "y")), (dx, ("dy", "w", "off", "out")),
                        (dw, ("dy", "x", "off", "out")), (save, ("x", "h", "ca")),
                        (back, ("dy", "ca", "dgate"))):
        for n in names:
            assert call(shape(), **{n: None}) == INVALID, (call, n)
    assert dx(shape(), dy2=P) == INVALID and dx(shape(), w2=P) == INVALID
    assert dw(shape(), acc=2) == INVALID
    assert dw(shape(rows=0), out=None) == INVALID        # written even without rows
    for call in (linear, dx):
        assert call(shape(), **{"ydt" if call is linear else "odt": E4M3}) == UNSUPPORTED


def test_no_rows_launch_nothing():
    s = shape(rows=0)
    assert linear(s, x=None, w=None, off=None, y=None) == 0
    assert dx(s, dy=None, out=None) == 0
    assert save(s, x=None) == 0 and back(s, dy=None) == 0


def test_workspaces():
    size = lambda name, *a: fn("moe_train", f"moe_{name}_workspace_size")(*a)
    s, big = shape(), shape(rows=4000, n=1000, k=1000)
    odd = shape(rows=4000, n=1001, k=1001)
    # operands that are read as they are need none; fp32 and odd ones do
    assert size("grouped_linear", big, BF16, 1) == size("grouped_linear_dw", big, BF16, 1) == 0
    assert size("grouped_linear_dx", big, BF16, 1, 1) == size("swiglu_checkpoint", big, BF16, 1) == 0
    for args in ((big, F32, 1), (odd, BF16, 1), (big, BF16, 0)):
        assert size("grouped_linear", *args) > 0 and size("swiglu_checkpoint", *args) > 0
        assert size("grouped_linear_dw", *args) > 0
        one, two = (size("grouped_linear_dx", args[0], args[1], t, args[2]) for t in (0, 1))
        assert two > one > 0
    assert size("swiglu_backward", s, BF16, 1) >= 10 * 2 * 4     # a term for 32 features of a row
    for name in ("grouped_linear", "grouped_linear_dw", "swiglu_checkpoint", "swiglu_backward"):
        assert size(name, shape(groups=0), BF16, 1) == size(name, s, E4M3, 1) == 0
    # three terms of so many rows are past 32-bit coordinates: nothing is copied
    assert size("grouped_linear", shape(rows=1 << 30, n=8, k=8), F32, 1) == 0
    # too small or off its alignment
    assert back(s, nws=16) == WORKSPACE and back(s, ws=None) == WORKSPACE
    assert back(s, ws=ctypes.c_void_p(0x1004)) == WORKSPACE
    assert save(s, dt=F32, nws=16) == WORKSPACE and save(s, dt=F32, ws=None) == WORKSPACE


def test_rows_refusals():
    sv, ld = fn("moe_train", "moe_checkpoint_rows"), fn("moe_train", "moe_restore_rows")
    assert sv(P, BF16, -1, 8, P, P, None) == INVALID
    assert sv(P, BF16, 1, 0, P, P, None) == INVALID
    assert sv(None, BF16, 1, 8, P, P, None) == INVALID
    assert sv(P, E4M3, 1, 8, P, P, None) == UNSUPPORTED
    assert sv(P, BF16, 1 << 31, 8, P, P, None) == UNSUPPORTED
    assert sv(None, BF16, 0, 8, None, None, None) == 0
    assert ld(P, P, 4, 8, None, 5, P, BF16, None, None) == INVALID   # more rows than there are
    assert ld(P, P, 4, 8, P, -1, P, BF16, None, None) == INVALID
    assert ld(P, P, 4, 8, P, 5, None, BF16, None, None) == INVALID
    assert ld(P, P, 4, 8, P, 5, P, E4M3, None, None) == UNSUPPORTED
    assert ld(None, None, 0, 8, None, 0, None, BF16, None, None) == 0


def test_reference_encoding_is_the_nearest_code():
    """The tests' own 8-bit form against torch's conversion."""
    v = R.normal(3, 40, 100, dtype=torch.float32) * torch.exp2(torch.linspace(-30, 30, 40))[:, None]
    e = R.scale_exps(v)
    codes, bad = R.e4m3_codes(v, e)
    s = torch.exp2(e.float() - 127).repeat_interleave(32, 1)[:, :100]
    assert not bad.any()
    assert torch.equal(codes, (v / s).to(torch.float8_e4m3fn).view(torch.uint8))
    assert (R.decode(codes, e) - v).abs().max() > 0


def test_reference_gradients_against_autograd():
    a, u, dh = (R.normal(i, 6, 10, dtype=torch.float32).double() for i in (1, 2, 3))
    gate = torch.rand(6, generator=torch.Generator().manual_seed(4)).double()
    a.requires_grad_(), u.requires_grad_(), gate.requires_grad_()
    (gate[:, None] * R.silu(a) * u * dh).sum().backward()
    vals, _ = R.swiglu_grads(a.detach(), u.detach(), dh, torch.zeros_like(dh), gate.detach(),
                             torch.float32)
    for got, want in zip(vals, (a.grad, u.grad, None, gate.grad)):
        if want is not None:
            assert (got - want).abs().max() < 1e-12


def test_training_rows_and_gather_refusals():
    from sparse_moe_layer_sum_b200._lib import MoECfg
    f, g = fn("moe_train", "moe_training_rows"), fn("moe_train", "moe_gather_rows")
    cfg = lambda **kw: ctypes.byref(MoECfg(*{**dict(
        dim=256, n_routed=16, n_groups=4, topk_groups=2, topk=4, inter=128, n_shared=1,
        route_scale=2.5, score_func=0, has_bias=1), **kw}.values()))
    call = lambda c, T=4, off=P, tok=P, out=P: f(c, T, off, tok, P, P, out, P, P, None, None)
    assert call(None) == INVALID and call(cfg(topk=0)) == INVALID and call(cfg(), T=-1) == INVALID
    assert call(cfg(n_shared=2)) == UNSUPPORTED and call(cfg(), T=1 << 29) == UNSUPPORTED
    assert call(cfg(), off=None) == INVALID and call(cfg(), tok=None) == INVALID
    assert call(cfg(), out=None) == INVALID
    assert g(P, BF16, 4, 8, None, 2, P, BF16, None, None) == INVALID
    assert g(P, BF16, 4, 0, P, 2, P, BF16, None, None) == INVALID
    assert g(None, BF16, 4, 8, P, 2, P, BF16, None, None) == INVALID
    assert g(P, E4M3, 4, 8, P, 2, P, BF16, None, None) == UNSUPPORTED
    assert g(P, BF16, 1 << 31, 8, P, 2, P, BF16, None, None) == UNSUPPORTED
    assert g(None, BF16, 4, 8, None, 0, None, BF16, None, None) == 0
