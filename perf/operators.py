"""Training operators of the experts: what is measured, and their plain forms.

Rows are expert-contiguous: group g owns rows offsets[g] .. offsets[g + 1] - 1.

    linear      y = x w[g]^T
    dx          dx = dy w[g], or the sum of two such products (the gate and the
                up projection share their input)
    dw          dw[g] = sum over the group's rows of dy^T x
    checkpoint  h = silu(x w1[g]^T) * (x w3[g]^T), with the two projections kept
                in 8 bits for the backward pass
    backward    from those 8 bits and dy: the projections' gradients, the gated
                hidden rows (the operand of w2's gradient) and the gates' gradients
    rows        a batch kept in 8 bits, and read back in expert order

The 8-bit format: e4m3 codes, one power-of-two scale for 32 values of a row, the
smallest with which the largest of them stays within 448.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the tiny block of the tests: 64 tokens, 4 of 16 experts; one small launch, latency counts
        dict(name="linear_tiny", op="linear", groups=16, rows=256, n=128, k=256, skew=0.0, dtype="bf16"),
        # first projection of a decode batch, 64 tokens by 8 experts: the weights' bytes count
        dict(name="linear_decode", op="linear", groups=256, rows=512, n=2048, k=7168, skew=0.0, dtype="bf16"),
        # first projection of a 4096-token batch: the tensor cores count
        dict(name="linear_prefill", op="linear", groups=256, rows=32768, n=2048, k=7168, skew=0.0, dtype="bf16"),
        # the single-precision configuration, with odd sizes
        dict(name="linear_f32_odd", op="linear", groups=17, rows=4099, n=517, k=1021, skew=0.5, dtype="f32"),
        # input gradient of both first projections, one of eight expert-parallel ranks
        dict(name="dx_shard", op="dx", groups=32, rows=4096, n=2048, k=7168, skew=0.3, dtype="bf16", dual=True),
        # gradient of the first projection's weights, the rank's share of 16384 tokens, uneven experts
        dict(name="dw_shard", op="dw", groups=32, rows=16384, n=2048, k=7168, skew=0.5, dtype="bf16", out="bf16"),
        # gradient of the second projection's weights in single precision, short groups
        dict(name="dw_f32_out", op="dw", groups=32, rows=4096, n=7168, k=2048, skew=0.3, dtype="bf16", out="f32"),
        # forward with its checkpoint, the tiny block
        dict(name="checkpoint_tiny", op="checkpoint", groups=16, rows=256, n=128, k=256, skew=0.0, dtype="bf16"),
        # forward with its checkpoint, one rank's share of 4096 tokens
        dict(name="checkpoint_shard", op="checkpoint", groups=32, rows=4096, n=2048, k=7168, skew=0.3, dtype="bf16"),
        # backward from the checkpoint, one rank's share of 16384 tokens
        dict(name="backward_shard", op="backward", groups=32, rows=16384, n=2048, k=7168, skew=0.5, dtype="bf16"),
        # backward from the checkpoint, small and ragged: some experts have no rows, sizes off every tile
        dict(name="backward_ragged", op="backward", groups=24, rows=333, n=200, k=264, skew=1.0, dtype="bf16"),
        # a 4096-token batch kept in 8 bits, read back in the order of 8 experts a token
        dict(name="rows_batch", op="rows", tokens=4096, rows=32768, k=7168, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "dx", "dw", "checkpoint", "backward", "rows"])
    dtype = "f32" if rng.random() < 0.15 else "bf16"
    if op == "rows":
        tokens = _log(rng, 1, 8192)
        return dict(op=op, tokens=tokens, rows=_log(rng, 1, 32768), k=_log(rng, 33, 7168), dtype=dtype)
    # a third of the widths is off every alignment (those are small models' widths), the others are
    # multiples of 8 or 64
    step = rng.choice([1, 8, 64])
    top = 600 if step == 1 else 2048 if dtype == "f32" else 7168
    n, k = (max(step, _log(rng, 64, t) // step * step) for t in (min(top, 4096), top))
    groups, rows = _log(rng, 1, 64), _log(rng, 1, 4096 if dtype == "f32" else 16384)
    rows = min(rows, int(1e11 / (n * k)))  # well within the largest listed case
    case = dict(op=op, groups=groups, rows=rows, n=n, k=k, skew=rng.choice([0.0, 0.3, 0.6]), dtype=dtype)
    if op == "dx":
        case["dual"] = rng.random() < 0.5
    if op == "dw":
        case["out"] = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
    return case


def _sizes(case, gen):
    """Rows of each group: a draw with replacement of an expert for every row."""
    G = case["groups"]
    p = torch.exp(case["skew"] * torch.randn(G, generator=gen))
    return torch.bincount(torch.multinomial(p, case["rows"], replacement=True, generator=gen), minlength=G)


def prepare(case, seed):
    dev = torch.device("cuda")
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype).mul_(std)

    s = dict(case=dict(case))
    if case["op"] == "rows":
        s["x"] = normal(case["tokens"], case["k"])
        s["index"] = torch.randint(case["tokens"], (case["rows"],), generator=gen, device=dev, dtype=torch.int32)
        return s
    G, R, N, K = case["groups"], case["rows"], case["n"], case["k"]
    sizes = _sizes(case, cpu)
    s["cap"] = int(sizes.max())
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(device=dev, dtype=torch.int32)
    op = case["op"]
    if op in ("linear", "checkpoint", "dw"):
        s["x"] = normal(R, K)
    if op in ("dx", "dw"):
        s["dy"] = normal(R, N)
    if op in ("linear", "dx"):
        s["w"] = normal(G, N, K, std=K ** -0.5)
    if op == "dx":
        s["dy2"], s["w2"] = (normal(R, N), normal(G, N, K, std=K ** -0.5)) if case["dual"] else (None, None)
    if op == "checkpoint":
        s["w1"], s["w3"] = normal(G, N, K, std=K ** -0.5), normal(G, N, K, std=K ** -0.5)
    if op == "backward":  # n: the hidden width, k: the model's width
        s["dy"] = normal(R, K)
        s["w2"] = normal(G, K, N, std=N ** -0.5)
        s["gate"] = torch.rand(R, generator=gen, device=dev) * 0.6 + 0.05
        s["a"], s["u"] = (_encode(normal(R, N, dtype=torch.float32)) for _ in range(2))
    return s


# ------------------------------------------------------------------ plain forms


def _pow2(biased):
    """2^(biased - 127) as float32, from its bits: biased 0 is the subnormal 2^-127."""
    b = biased.to(torch.int32)
    return torch.where(b > 0, b << 23, 1 << 22).view(torch.float32)


def _encode(v):
    """(e4m3 codes [rows, n] as uint8, biased scale exponents [rows, ceil(n / 32)] as uint8)."""
    rows, n = v.shape
    b = torch.nn.functional.pad(v, (0, -n % 32)).reshape(rows, -1, 32)
    amax = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(2)
    m, e = torch.frexp(amax)                        # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875), -127).clamp_min(-127)
    exps = (e + 127).to(torch.uint8)
    code = (b / _pow2(exps)[:, :, None]).to(torch.float8_e4m3fn)
    return code.reshape(rows, -1)[:, :n].contiguous().view(torch.uint8), exps


def _decode(code, exps):
    scale = _pow2(exps).repeat_interleave(32, 1)[:, : code.shape[1]]
    return code.view(torch.float8_e4m3fn).float() * scale


def _place(s, rows):
    """Group of each row, and its place in the group."""
    off = s["offsets"].long()
    p = torch.arange(rows, device=off.device)
    g = torch.searchsorted(off[1:], p, right=True)
    return g, p - off[g]


def _pad(s, v, at):
    """[groups, longest group, width], zeros behind a group's rows."""
    out = torch.zeros(s["offsets"].numel() - 1, s["cap"], v.shape[1], dtype=torch.float32, device=v.device)
    out[at] = v.float()
    return out


def _plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    op = c["op"]
    if op == "rows":
        return _decode(*_encode(s["x"].float()))[s["index"].long()].to(dt)
    at = _place(s, c["rows"])
    if op == "linear":
        return torch.matmul(_pad(s, s["x"], at), s["w"].float().transpose(1, 2))[at].to(dt)
    if op == "dx":
        dx = torch.matmul(_pad(s, s["dy"], at), s["w"].float())
        if c["dual"]:
            dx += torch.matmul(_pad(s, s["dy2"], at), s["w2"].float())
        return dx[at].to(dt)
    if op == "dw":
        return torch.matmul(_pad(s, s["dy"], at).transpose(1, 2), _pad(s, s["x"], at)).to(DTYPES[c["out"]])
    if op == "checkpoint":
        x = _pad(s, s["x"], at)
        a = torch.matmul(x, s["w1"].float().transpose(1, 2))[at]
        u = torch.matmul(x, s["w3"].float().transpose(1, 2))[at]
        h = (a * torch.sigmoid(a) * u).to(dt)
        return _held(h, _encode(a), _encode(u))
    dh = torch.matmul(_pad(s, s["dy"], at), s["w2"].float())[at]
    a, u, g = _decode(*s["a"]), _decode(*s["u"]), s["gate"][:, None]
    sig = torch.sigmoid(a)
    h = a * sig * u
    return [(g * dh * u * sig * (1 + a * (1 - sig))).to(dt), (g * dh * a * sig).to(dt), (g * h).to(dt), (dh * h).sum(1)]


def _held(h, a, u):
    """What an 8-bit checkpoint holds, as numbers: the codes' values and the scales'."""
    return [h] + [v for code, exps in (a, u) for v in (code.view(torch.float8_e4m3fn), exps.view(torch.float8_e8m0fnu))]


# ----------------------------------------------------------------------- passes


def run(s):
    if not own:
        return _plain(s)
    import sparse_moe_layer_sum_b200 as moe

    c = s["case"]
    op = c["op"]
    if op == "rows":
        return moe.restore_rows(moe.checkpoint_rows(s["x"]), s["index"], dtype=s["x"].dtype)
    if op == "linear":
        return moe.grouped_linear(s["x"], s["w"], s["offsets"])
    if op == "dx":
        return moe.grouped_linear_dx(s["dy"], s["w"], s["offsets"], dy2=s["dy2"], w2=s["w2"])
    if op == "dw":
        return moe.grouped_linear_dw(s["dy"], s["x"], s["offsets"], out_dtype=DTYPES[c["out"]])
    if op == "checkpoint":
        h, a, u = moe.swiglu_checkpoint(s["x"], s["w1"], s["w3"], s["offsets"])
        return _held(h, (a.codes, a.exps), (u.codes, u.exps))
    a, u = (moe.Checkpoint(*s[v]) for v in "au")
    return list(moe.swiglu_backward(s["dy"], s["w2"], a, u, s["offsets"], gate=s["gate"]))


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op, R, K = case["op"], case["rows"], case["k"]
    if op == "rows":
        T = case["tokens"]
        seen = T * (1 - (1 - 1 / T) ** R)  # distinct rows that are read back, expected
        kept = K + -(-K // 32)
        return {"bytes": T * (K * e + kept) + seen * kept + R * (K * e + 4), "flops": 2 * T * K + R * K}
    G, N = case["groups"], case["n"]
    live = G * (1 - (1 - 1 / G) ** R)      # groups with rows, expected
    w = live * N * K * e
    if op == "linear":
        return {"bytes": R * (N + K) * e + w, "flops": 2 * R * N * K}
    if op == "dx":
        t = 2 if case["dual"] else 1
        return {"bytes": R * (t * N + K) * e + t * w, "flops": 2 * t * R * N * K}
    if op == "dw":
        return {"bytes": R * (N + K) * e + G * N * K * (4 if case["out"] == "f32" else 2), "flops": 2 * R * N * K}
    kept = 2 * R * (N + -(-N // 32))
    if op == "checkpoint":
        return {"bytes": R * (K + N) * e + 2 * w + kept, "flops": 4 * R * N * K}
    return {"bytes": R * (K + 3 * N) * e + w + kept + 8 * R, "flops": 2 * R * N * K + 12 * R * N}


# ------------------------------------------------------------- 64 bits, by group


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64

    def two(e):  # 2^e for whole numbers e of the normal range, from its bits
        return ((e.to(torch.int64) + 1023) << 52).view(f64)

    def values(code, exps):
        v = code.view(torch.float8_e4m3fn).to(f64)
        for b in range(exps.shape[1]):
            v[:, 32 * b:32 * b + 32] *= two(exps[:, b:b + 1].to(torch.int64) - 127)
        return v

    def held(v):
        """(codes' values, scales) of the rows of v."""
        code, scale = torch.empty_like(v), []
        for b in range(-(-v.shape[1] // 32)):
            t = v[:, 32 * b:32 * b + 32]
            top = t.abs().amax(1, keepdim=True)
            sc = two(torch.ceil(torch.log2(top / 448)).clamp_min(-127))
            sc = torch.where(top > 0, torch.where(top / sc * 2 <= 448, sc / 2, torch.where(top / sc > 448, sc * 2, sc)), 2.0 ** -127)
            q = t / sc
            step = two(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
            code[:, 32 * b:32 * b + 32] = torch.round(q / step) * step  # half to even, as e4m3 rounds
            scale.append(sc)
        return code, torch.cat(scale, 1)

    if op == "rows":
        code, scale = held(s["x"].to(f64))
        return (code * scale.repeat_interleave(32, 1)[:, : code.shape[1]])[s["index"].long()]
    off = s["offsets"].tolist()
    parts = []
    for g, (lo, hi) in enumerate(zip(off, off[1:])):
        t = {k: s[k][lo:hi].to(f64) for k in ("x", "dy", "dy2") if s.get(k) is not None}
        w = {k: s[k][g].to(f64) for k in ("w", "w1", "w2", "w3") if s.get(k) is not None}
        if op == "linear":
            parts.append([t["x"] @ w["w"].T])
        elif op == "dx":
            parts.append([t["dy"] @ w["w"] + (t["dy2"] @ w["w2"] if case["dual"] else 0.0)])
        elif op == "dw":
            parts.append([(t["dy"].T @ t["x"])[None]])
        elif op == "checkpoint":
            a, u = t["x"] @ w["w1"].T, t["x"] @ w["w3"].T
            parts.append([a / (1 + torch.exp(-a)) * u, *held(a), *held(u)])
        else:
            a, u = (values(s[v][0][lo:hi], s[v][1][lo:hi]) for v in "au")
            gate = s["gate"][lo:hi, None].to(f64)
            dh, sig = t["dy"] @ w["w2"], 1 / (1 + torch.exp(-a))
            parts.append([gate * dh * u * (sig + a * sig * (1 - sig)), gate * dh * a * sig, gate * a * sig * u,
                          (dh * a * sig * u).sum(1)])
    out = [torch.cat(p) for p in zip(*parts)]
    return out if op in ("checkpoint", "backward") else out[0]
