"""Python binding of the experts' training operators (moe_train).

Argument marshalling only, as in moe.py.  Row buffers are expert-contiguous:
group g owns rows offsets[g] .. offsets[g + 1] - 1, the order dispatch_build
produces.  Every function allocates its outputs (or takes them as `out`, apart
from the operands), enqueues on the current stream of the operands' device and
does not synchronise; rows outside the groups are left as they were.  Autograd
does not see these calls, as it does not see the rest of the package: no result
requires a gradient, whatever the operands do, and the backward pass is called
by name.

    y  = grouped_linear(x, w, offsets)                    # y = x w^T, by group
    dx = grouped_linear_dx(dy, w, offsets)                # dx = dy w
    dw = grouped_linear_dw(dy, x, offsets)                # dw = dy^T x
    h, a, u = swiglu_checkpoint(x, w1, w3, offsets)       # a, u kept in 8 bits
    da, du, hg, dgate = swiglu_backward(dy, w2, a, u, offsets, gate=gate)

Together they train the experts of a block on the routing of a batch:

    weights, indices, _ = router_forward(shape, x, w_r, bias)
    _, offsets, sorted_token, slot_of = dispatch_build(shape, indices)
    y, saved = experts_training_forward(shape, params, x, weights, offsets, sorted_token, slot_of)
    grads = experts_training_backward(shape, params, saved, dy)
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import MoEGroupedShape, check, fn
from .moe import BlockParams, BlockShape, _ptr, combine

_DT = {torch.float32: _lib.DTYPES["f32"], torch.bfloat16: _lib.DTYPES["bf16"]}
SCALE_BLOCK = 32  # values of a row that share a scale


@dataclass
class Checkpoint:
    """Rows kept in 8 bits: e4m3 codes [rows, k] (uint8) and one biased
    power-of-two exponent for 32 values, exps [rows, ceil(k / 32)] (uint8);
    value = e4m3(code) * 2^(exp - 127)."""

    codes: torch.Tensor
    exps: torch.Tensor

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.exps.numel()


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _check(first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    """The CUDA device of all of them (an index)."""
    dev = first.get_device()
    if dev < 0 or not first.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    for t in others:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and on one CUDA device")
    return dev


_fn: dict = {}  # entry points of moe_train, looked up once


def _entry(sym: str):
    f = _fn.get(sym)
    if f is None:
        f = _fn[sym] = fn("moe_train", sym)
    return f


def _call(dev: int, sym: str, *args) -> None:
    """Call `sym` of moe_train with `dev` current, on its current stream.  (The
    raw stream handle is read directly: torch.cuda.current_stream() alone takes
    as long as the rest of a call.)"""
    f = _entry(sym)
    if dev == torch._C._cuda_getDevice():
        st = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        check(st, sym)


def _groups(offsets: torch.Tensor) -> int:
    n = offsets.shape
    if offsets.dtype != torch.int32 or len(n) != 1 or n[0] < 2:
        raise ValueError("offsets must be int32 [groups + 1]")
    return n[0] - 1


def _dtype(t: torch.Tensor, *others: torch.Tensor) -> int:
    d = t.dtype
    dt = _DT.get(d)
    if dt is None:
        raise ValueError("operands must be bf16 or fp32")
    for o in others:
        if o.dtype != d:
            raise ValueError("operands must have one dtype")
    return dt


def _apart(out: torch.Tensor, operands) -> None:
    """Refuse an `out` that shares memory with what the call reads: blocks that
    finish early would overwrite operands of the others."""
    lo = out.data_ptr()
    hi = lo + out.numel() * out.element_size()
    for t in operands:
        if t is None or lo == hi:
            continue
        at = t.data_ptr()
        if at < hi and lo < at + t.numel() * t.element_size():
            raise ValueError("out must not share memory with an operand")


def _out(out, out_dtype, dtype, dev: int, operands, *shape: int):
    """(`out` or a new tensor, its dtype code) for a result of `shape`, in
    out_dtype or else `dtype`, apart from the operands."""
    if out is None:
        dtype = out_dtype or dtype
    elif out.shape != shape or (out_dtype or out.dtype) != out.dtype:
        raise ValueError("out has another shape or dtype")
    else:
        dtype = out.dtype
        _apart(out, operands)
    dt = _DT.get(dtype)
    if dt is None:
        raise ValueError("outputs must be bf16 or fp32")
    return (torch.empty(*shape, dtype=dtype, device=dev) if out is None else out), dt


def _status(status: Optional[torch.Tensor]) -> Optional[int]:
    if status is None:
        return None
    _need(status.dtype == torch.int32 and status.numel() >= 1, "status must be int32")
    return status.data_ptr()


_plans: dict = {}  # (moe_grouped_shape, workspace bytes) by what they depend on


def _plan(sym: str, dev: int, G: int, n: int, k: int, rows: int, dt: int, operands, *flags: int):
    """(shape, workspace or None, its address or None, its bytes) for a call whose
    workspace `sym` states; operands are the tensors its alignment goes by."""
    aligned = 1
    for t in operands:
        if t.data_ptr() & 15:
            aligned = 0
    key = (sym, G, n, k, rows, dt, aligned, flags)
    p = _plans.get(key)
    if p is None:
        if len(_plans) > 4096:
            _plans.clear()
        shape = ctypes.byref(MoEGroupedShape(G, n, k, rows))
        p = _plans[key] = (shape, _entry(sym)(shape, dt, *flags, aligned))
    shape, need = p
    if not need:
        return shape, None, None, 0
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    return shape, ws, ws.data_ptr(), need


def grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *,
                   out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                   status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_grouped_linear: y[p] = x[p] w[g]^T for the rows p of each group g.
    x [rows, k], w [groups, n, k] -> y [rows, n] (x's dtype unless out_dtype)."""
    dev = _check(x, w, offsets, out, status)
    G = _groups(offsets)
    xs, wsh = x.shape, w.shape
    if len(xs) != 2 or len(wsh) != 3 or wsh[0] != G or wsh[2] != xs[1]:
        raise ValueError("x must be [rows, k] and w [groups, n, k]")
    dt = _dtype(x, w)
    (rows, k), n = xs, wsh[1]
    out, odt = _out(out, out_dtype, x.dtype, dev, (x, w, offsets), rows, n)
    shape, ws, at, nws = _plan("moe_grouped_linear_workspace_size", dev, G, n, k, rows, dt, (x, w))
    _call(dev, "moe_grouped_linear", shape, x.data_ptr(), dt, w.data_ptr(), offsets.data_ptr(),
          out.data_ptr(), odt, at, nws, _status(status))
    return out


def grouped_linear_dx(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *,
                      dy2: Optional[torch.Tensor] = None, w2: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                      status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_grouped_linear_dx: dx[p] = dy[p] w[g] (+ dy2[p] w2[g], in one sum).
    dy [rows, n], w [groups, n, k] -> dx [rows, k] (dy's dtype unless out_dtype)."""
    dev = _check(dy, w, dy2, w2, offsets, out, status)
    G = _groups(offsets)
    ys, wsh = dy.shape, w.shape
    if len(ys) != 2 or len(wsh) != 3 or wsh[0] != G or wsh[1] != ys[1]:
        raise ValueError("dy must be [rows, n] and w [groups, n, k]")
    two = dy2 is not None
    _need(two == (w2 is not None), "dy2 and w2 come together")
    if two:
        _need(dy2.shape == ys and w2.shape == wsh, "dy2 and w2 must match dy and w")
    operands = (dy, w, dy2, w2) if two else (dy, w)
    dt = _dtype(*operands)
    (rows, n), k = ys, wsh[2]
    out, odt = _out(out, out_dtype, dy.dtype, dev, (*operands, offsets), rows, k)
    shape, ws, at, nws = _plan("moe_grouped_linear_dx_workspace_size", dev, G, n, k, rows, dt, operands,
                               int(two))
    _call(dev, "moe_grouped_linear_dx", shape, dy.data_ptr(), dt, w.data_ptr(), _ptr(dy2), _ptr(w2),
          offsets.data_ptr(), out.data_ptr(), odt, at, nws, _status(status))
    return out


def grouped_linear_dw(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, *,
                      out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                      accumulate: bool = False,
                      status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_grouped_linear_dw: dw[g] = sum over the group's rows of dy^T x, added
    to `out` with accumulate.  dy [rows, n], x [rows, k] -> dw [groups, n, k]
    (dy's dtype unless out_dtype); zero for a group without rows."""
    dev = _check(dy, x, offsets, out, status)
    G = _groups(offsets)
    ys, xs = dy.shape, x.shape
    if len(ys) != 2 or len(xs) != 2 or xs[0] != ys[0]:
        raise ValueError("dy must be [rows, n] and x [rows, k]")
    _need(out is not None or not accumulate, "accumulate needs out")
    dt = _dtype(dy, x)
    (rows, n), k = ys, xs[1]
    out, odt = _out(out, out_dtype, dy.dtype, dev, (dy, x, offsets), G, n, k)
    shape, ws, at, nws = _plan("moe_grouped_linear_dw_workspace_size", dev, G, n, k, rows, dt, (dy, x))
    _call(dev, "moe_grouped_linear_dw", shape, dy.data_ptr(), dt, x.data_ptr(), offsets.data_ptr(),
          out.data_ptr(), odt, int(accumulate), at, nws, _status(status))
    return out


def _blocks(k: int) -> int:
    return -(-k // SCALE_BLOCK)


def _empty_ckpt(rows: int, k: int, dev: int) -> Checkpoint:
    u8 = torch.uint8
    return Checkpoint(torch.empty(rows, k, dtype=u8, device=dev),
                      torch.empty(rows, _blocks(k), dtype=u8, device=dev))


def _check_ckpt(c: Checkpoint, rows: int, k: int) -> None:
    codes, exps = c.codes, c.exps
    if (codes.dtype != torch.uint8 or exps.dtype != torch.uint8 or codes.shape != (rows, k)
            or exps.shape != (rows, _blocks(k))):
        raise ValueError("a checkpoint holds uint8 codes [rows, k] and exps [rows, ceil(k / 32)]")


def checkpoint_rows(src: torch.Tensor) -> Checkpoint:
    """moe_checkpoint_rows: src [rows, k] (bf16 or fp32) kept in 8 bits."""
    dev = _check(src)
    _need(src.dim() == 2, "src must be [rows, k]")
    dt = _dtype(src)
    rows, k = src.shape
    c = _empty_ckpt(rows, k, dev)
    _call(dev, "moe_checkpoint_rows", src.data_ptr(), dt, rows, k, c.codes.data_ptr(),
          c.exps.data_ptr())
    return c


def restore_rows(ckpt: Checkpoint, index: Optional[torch.Tensor] = None, *,
                 dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_restore_rows: the stored rows [n, k], row index[i] at place i (int32;
    every row in order without index)."""
    dev = _check(ckpt.codes, ckpt.exps, index, out, status)
    _need(ckpt.codes.dim() == 2, "codes must be [rows, k]")
    rows, k = ckpt.codes.shape
    _check_ckpt(ckpt, rows, k)
    if index is not None:
        _need(index.dtype == torch.int32 and index.dim() == 1, "index must be int32 [n]")
    n = rows if index is None else index.numel()
    out, odt = _out(out, None, dtype, dev, (ckpt.codes, ckpt.exps, index), n, k)
    _call(dev, "moe_restore_rows", ckpt.codes.data_ptr(), ckpt.exps.data_ptr(), rows, k,
          _ptr(index), n, out.data_ptr(), odt, _status(status))
    return out


def swiglu_checkpoint(x: torch.Tensor, w1: torch.Tensor, w3: torch.Tensor, offsets: torch.Tensor, *,
                      status: Optional[torch.Tensor] = None):
    """moe_swiglu_checkpoint: (h, a, u) with h = silu(x w1^T) * (x w3^T) by group
    [rows, n] and the two projections as Checkpoints.  x [rows, k],
    w1, w3 [groups, n, k]."""
    dev = _check(x, w1, w3, offsets, status)
    G = _groups(offsets)
    xs, wsh = x.shape, w1.shape
    if len(xs) != 2 or len(wsh) != 3 or wsh[0] != G or wsh[2] != xs[1] or w3.shape != wsh:
        raise ValueError("x must be [rows, k], w1 and w3 [groups, n, k]")
    operands = (x, w1, w3)
    dt = _dtype(*operands)
    (rows, k), n = xs, wsh[1]
    h = torch.empty(rows, n, dtype=x.dtype, device=dev)
    a, u = _empty_ckpt(rows, n, dev), _empty_ckpt(rows, n, dev)
    shape, ws, at, nws = _plan("moe_swiglu_checkpoint_workspace_size", dev, G, n, k, rows, dt, operands)
    _call(dev, "moe_swiglu_checkpoint", shape, x.data_ptr(), dt, w1.data_ptr(),
          w3.data_ptr(), offsets.data_ptr(), h.data_ptr(), a.codes.data_ptr(), a.exps.data_ptr(),
          u.codes.data_ptr(), u.exps.data_ptr(), at, nws, _status(status))
    return h, a, u


def swiglu_backward(dy: torch.Tensor, w2: torch.Tensor, a: Checkpoint, u: Checkpoint,
                    offsets: torch.Tensor, *, gate: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None):
    """moe_swiglu_backward: (da, du, hg, dgate) of gate * (h w2^T) for the h of a
    checkpoint.  dy [rows, k], w2 [groups, k, n], gate [rows] fp32 (1 without)
    -> da, du, hg [rows, n] in dy's dtype, dgate [rows] fp32."""
    dev = _check(dy, w2, a.codes, a.exps, u.codes, u.exps, gate, offsets, status)
    G = _groups(offsets)
    ys, wsh = dy.shape, w2.shape
    if len(ys) != 2 or len(wsh) != 3 or wsh[0] != G or wsh[1] != ys[1]:
        raise ValueError("dy must be [rows, k] and w2 [groups, k, n]")
    dt = _dtype(dy, w2)
    (rows, k), n = ys, wsh[2]
    _check_ckpt(a, rows, n)
    _check_ckpt(u, rows, n)
    if gate is not None:
        _need(gate.dtype == torch.float32 and tuple(gate.shape) == (rows,), "gate must be fp32 [rows]")
    dtype = dy.dtype
    da, du, hg = (torch.empty(rows, n, dtype=dtype, device=dev) for _ in range(3))
    dgate = torch.empty(rows, dtype=torch.float32, device=dev)
    shape, ws, at, nws = _plan("moe_swiglu_backward_workspace_size", dev, G, n, k, rows, dt, (dy, w2))
    _call(dev, "moe_swiglu_backward", shape, dy.data_ptr(), dt, w2.data_ptr(),
          a.codes.data_ptr(), a.exps.data_ptr(), u.codes.data_ptr(), u.exps.data_ptr(), _ptr(gate),
          offsets.data_ptr(), da.data_ptr(), du.data_ptr(), hg.data_ptr(), dgate.data_ptr(),
          at, nws, _status(status))
    return da, du, hg, dgate


def gather_rows(src: torch.Tensor, index: torch.Tensor, *, dtype: Optional[torch.dtype] = None,
                status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_gather_rows: src[index] for src [rows, k] and index [n] int32, in
    `dtype` (src's own without)."""
    dev = _check(src, index, status)
    _need(src.dim() == 2 and index.dtype == torch.int32 and index.dim() == 1,
          "src must be [rows, k] and index int32 [n]")
    dt = _dtype(src)
    (rows, k), n = src.shape, index.numel()
    out, odt = _out(None, dtype, src.dtype, dev, (), n, k)
    _call(dev, "moe_gather_rows", src.data_ptr(), dt, rows, k, index.data_ptr(), n, out.data_ptr(),
          odt, _status(status))
    return out


def training_rows(shape: BlockShape, weights: torch.Tensor, offsets: torch.Tensor,
                  sorted_token: torch.Tensor, slot_of: torch.Tensor, *,
                  status: Optional[torch.Tensor] = None):
    """moe_training_rows: (row_token, row_gate, group_offsets) of a batch's
    routed rows followed by the shared expert's."""
    dev = _check(weights, offsets, sorted_token, slot_of, status)
    T, k = weights.shape
    _need(k == shape.topk and weights.dtype == torch.float32, "weights must be fp32 [T, topk]")
    _need(offsets.dtype == sorted_token.dtype == slot_of.dtype == torch.int32
          and offsets.numel() == shape.n_routed + 1
          and sorted_token.numel() == slot_of.numel() == T * k,
          "offsets, sorted_token and slot_of must be dispatch_build's")
    R = T * (k + shape.n_shared)
    row_token = torch.empty(R, dtype=torch.int32, device=dev)
    row_gate = torch.empty(R, dtype=torch.float32, device=dev)
    group_offsets = torch.empty(shape.n_routed + shape.n_shared + 1, dtype=torch.int32, device=dev)
    cfg = shape.cfg()
    _call(dev, "moe_training_rows", ctypes.byref(cfg), T, offsets.data_ptr(), sorted_token.data_ptr(),
          slot_of.data_ptr(), weights.data_ptr(), row_token.data_ptr(), row_gate.data_ptr(),
          group_offsets.data_ptr(), _status(status))
    return row_token, row_gate, group_offsets


@dataclass
class SavedExperts:
    """What experts_training_forward leaves for the backward pass: the batch
    and the two projections in 8 bits, and the routing's row lists."""

    x: Checkpoint
    a: Checkpoint
    u: Checkpoint
    row_token: torch.Tensor
    row_gate: torch.Tensor
    group_offsets: torch.Tensor
    slot_of: torch.Tensor
    dtype: torch.dtype

    @property
    def nbytes(self) -> int:
        return self.x.nbytes + self.a.nbytes + self.u.nbytes


@dataclass
class ExpertGrads:
    """Gradients of one batch: dx [T, dim] fp32 (through the experts; the
    router's share is not in it), dgates [T, topk] fp32, and the weights'
    gradients, stacked as the weights are."""

    dx: torch.Tensor
    dgates: torch.Tensor
    dw1: torch.Tensor
    dw3: torch.Tensor
    dw2: torch.Tensor


def _token_sums(shape: BlockShape, weights, slot_of, rows, status) -> torch.Tensor:
    """moe_combine of the routed rows, then the shared expert's."""
    n = weights.numel()
    with torch.cuda.device(rows.device):
        return combine(shape, weights, slot_of, rows[:n], rows[n:] if shape.n_shared else None,
                       status=status)


def experts_training_forward(shape: BlockShape, params: BlockParams, x: torch.Tensor,
                             weights: torch.Tensor, offsets: torch.Tensor,
                             sorted_token: torch.Tensor, slot_of: torch.Tensor, *,
                             status: Optional[torch.Tensor] = None):
    """(y [T, dim] fp32, SavedExperts) of the routed experts and the shared one
    for x [T, dim], with the routing of router_forward and dispatch_build.
    Weights in x's dtype (bf16 or fp32), all experts' of the shape: the shards
    of expert-parallel ranks are refused.  y is the ordered sum of moe_combine,
    bit-reproducible.  x and the projections are kept in 8 bits, with fp32
    weights too."""
    _need(x.dim() == 2 and x.shape[1] == shape.dim, "x must be [T, dim]")
    _need(params.w1.dtype == x.dtype and x.dtype in _DT, "training takes weights in x's dtype")
    T, k = x.shape[0], shape.topk
    _need(tuple(weights.shape) == (T, k) and sorted_token.numel() == slot_of.numel() == T * k,
          "the routing is not that of x's T rows")
    row_token, row_gate, group_offsets = training_rows(shape, weights, offsets, sorted_token, slot_of,
                                                       status=status)
    rows = gather_rows(x, row_token, status=status)
    h, a, u = swiglu_checkpoint(rows, params.w1, params.w3, group_offsets, status=status)
    o = grouped_linear(h, params.w2, group_offsets, out_dtype=torch.float32, status=status)
    y = _token_sums(shape, weights, slot_of, o, status)
    return y, SavedExperts(checkpoint_rows(x), a, u, row_token, row_gate, group_offsets, slot_of,
                           x.dtype)


def experts_training_backward(shape: BlockShape, params: BlockParams, saved: SavedExperts,
                              dy: torch.Tensor, *, grad_dtype: torch.dtype = torch.float32,
                              accumulate: Optional[ExpertGrads] = None,
                              status: Optional[torch.Tensor] = None) -> ExpertGrads:
    """Gradients of experts_training_forward for dy [T, dim] (fp32 or the
    weights' dtype).  With `accumulate` the weights' gradients are added to its
    dw1, dw3 and dw2; otherwise they are new tensors of grad_dtype."""
    T, k = saved.x.codes.shape[0], shape.topk
    _need(tuple(dy.shape) == (T, shape.dim), "dy must be [T, dim]")
    # (combine and the gathers below go by T, topk and the saved lists together)
    _need(saved.slot_of.numel() == T * k
          and saved.row_token.numel() == saved.row_gate.numel() == T * (k + shape.n_shared)
          and saved.group_offsets.numel() == shape.n_routed + shape.n_shared + 1,
          "saved is not of a batch of this shape")
    if accumulate is not None:  # all of them before any is added to
        for name in ("w1", "w3", "w2"):
            t, w = getattr(accumulate, "d" + name), getattr(params, name)
            _need(t.shape == w.shape and t.dtype in _DT and t.device == w.device and t.is_contiguous(),
                  "accumulate must hold gradients of the weights' shapes")
    st = dict(status=status)
    off = saved.group_offsets
    dyr = gather_rows(dy, saved.row_token, dtype=saved.dtype, **st)
    da, du, hg, dgate = swiglu_backward(dyr, params.w2, saved.a, saved.u, off, gate=saved.row_gate, **st)

    def dw(d, rows, name):
        out = getattr(accumulate, name) if accumulate is not None else None
        return grouped_linear_dw(d, rows, off, out=out, out_dtype=None if out is not None else grad_dtype,
                                 accumulate=out is not None, **st)

    dw2 = dw(dyr, hg, "dw2")
    rows = restore_rows(saved.x, saved.row_token, dtype=saved.dtype, **st)
    dw1, dw3 = dw(da, rows, "dw1"), dw(du, rows, "dw3")
    dxr = grouped_linear_dx(da, params.w1, off, dy2=du, w2=params.w3, out_dtype=torch.float32, **st)
    # the tokens' rows summed in slot order, the shared expert's last
    ones = torch.ones(T, k, dtype=torch.float32, device=dy.device)
    dx = _token_sums(shape, ones, saved.slot_of, dxr, status)
    dgates = gather_rows(dgate[:T * k].view(-1, 1), saved.slot_of.view(-1), **st).view(T, k)
    return ExpertGrads(dx, dgates, dw1, dw3, dw2)
