"""64-bit CPU forms of the training operators, and the inputs and error bounds
the GPU tests share.  Test infrastructure only; no code of the package.

Bounds are per element.  A product's sum of K terms t_i is kept in fp32, where
each addition is off by at most one step (2^-23) of a partial sum that is at
most S = sum |t_i|; bf16 and fp32 products enter with at most one more step:
    E = (K + 1) * 2^-23 * S
and the result is rounded once, by half a step of its type:
    |y - exact| <= E + half * (|exact| + E)
"""
import math

import torch

F64 = torch.float64
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
ULP = 2.0 ** -23


def offsets_of(sizes, first=0):
    o = [first]
    for s in sizes:
        o.append(o[-1] + s)
    return o


def normal(seed, *shape, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float32) * std).to(dtype)


def groups(off):
    return [(g, slice(a, b)) for g, (a, b) in enumerate(zip(off, off[1:]))]


def linear(x, w, off):
    """(y, E): x [rows, k], w [G, n, k]; rows outside the groups are zero."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=F64)
    e = torch.zeros_like(y)
    for g, r in groups(off):
        xd, wd = x[r].to(F64), w[g].to(F64)
        y[r] = xd @ wd.T
        e[r] = (x.shape[1] + 1) * ULP * (xd.abs() @ wd.abs().T)
    return y, e


def dx(dy, w, off, dy2=None, w2=None):
    t = [linear(a, b.transpose(1, 2), off) for a, b in ((dy, w), (dy2, w2)) if a is not None]
    if len(t) == 1:
        return t[0]
    return t[0][0] + t[1][0], 2 * (t[0][1] + t[1][1])   # 2 K terms of the summed magnitudes


def dw(dy, x, off):
    y = torch.zeros(len(off) - 1, dy.shape[1], x.shape[1], dtype=F64)
    e = torch.zeros_like(y)
    for g, r in groups(off):
        a, b = dy[r].to(F64), x[r].to(F64)
        y[g] = a.T @ b
        e[g] = (a.shape[0] + 1) * ULP * (a.abs().T @ b.abs())
    return y, e


def scale_exps(v):
    """Biased scale exponents [rows, ceil(n / 32)] by the definition: the
    smallest e >= 0 with amax <= 448 * 2^(e - 127)."""
    rows, n = v.shape
    out = torch.zeros(rows, math.ceil(n / 32), dtype=torch.uint8)
    for b in range(out.shape[1]):
        t = v[:, 32 * b:32 * b + 32].to(F64)
        top = torch.where(torch.isfinite(t), t.abs(), 0.0).amax(1)
        for i, m in enumerate(top.tolist()):
            e = 0
            if m > 0:
                e = max(0, math.frexp(m)[1] - 9 + 127 - 1)
                while m > 448 * 2.0 ** (e - 127):
                    e += 1
            out[i, b] = e
    return out


def e4m3_codes(v, exps):
    """Codes by a search of the 256 codes for the nearest value (ties to the
    even code); non-finite values to NaN."""
    table = torch.arange(128, dtype=torch.uint8).view(torch.float8_e4m3fn).to(F64)[:127]
    s = torch.pow(2.0, exps.to(F64) - 127).repeat_interleave(32, 1)[:, : v.shape[1]]
    q = v.to(F64) / s
    hi = torch.searchsorted(table, q.abs().contiguous()).clamp(1, 126)
    dlo, dhi = q.abs() - table[hi - 1], table[hi] - q.abs()
    code = torch.where((dlo < dhi) | ((dlo == dhi) & (hi % 2 == 1)), hi - 1, hi)
    code = code + torch.where(torch.signbit(q), 128, 0)
    bad = ~torch.isfinite(v.to(F64))
    return code.to(torch.uint8), bad


def decode(codes, exps):
    s = torch.pow(2.0, exps.to(F64) - 127).repeat_interleave(32, 1)[:, : codes.shape[1]]
    return codes.view(torch.float8_e4m3fn).to(F64) * s


def silu(a):
    return a / (1 + torch.exp(-a))


def sigmoid_rel(a, dtype):
    """Relative error of the kernels' sigmoid.  bf16 results use the hardware
    exponential (2 + 1.173 |a| steps by the CUDA guide's table) and reciprocal
    (2 steps); fp32 ones expf (1 step) and a division."""
    steps = 5 + 1.2 * a.abs() if dtype == torch.bfloat16 else 4.0 + 0 * a
    return steps * ULP


def swiglu_grads(a, u, dh, e_dh, gate, dtype):
    """((da, du, hg, dgate), their bounds before the last rounding)."""
    s = 1 / (1 + torch.exp(-a))
    g = gate[:, None]
    h, ds = a * s * u, s * (1 + a * (1 - s))
    vals = (g * dh * u * ds, g * dh * a * s, g * h, (dh * h).sum(1))
    r = sigmoid_rel(a, dtype) + 8 * ULP
    # ds = s + a s (1 - s): an error of s r moves it by at most s r (1 + 2 |a|)
    b_da = (g * u).abs() * (e_dh * ds.abs() + (dh.abs() + e_dh) * s * (1 + 2 * a.abs()) * r)
    b_du = (g * a * s).abs() * (e_dh + (dh.abs() + e_dh) * r)
    b_hg = (g * h).abs() * r
    n = a.shape[1]
    b_dg = ((e_dh + dh.abs() * (r + (n + 1) * ULP)) * h.abs()).sum(1)
    return vals, (b_da, b_du, b_hg, b_dg)


def assert_close(got, want, err, what=""):
    half = HALF[got.dtype]
    d = (got.to(F64).cpu() - want).abs()
    # 2^-133 / 2: bf16's smallest step near zero
    tol = err + half * (want.abs() + err) + 2.0 ** -134
    bad = ~(d <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((d / tol).nan_to_num(nan=9e9).max()):.3g} of the bound")
