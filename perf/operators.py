"""What the layer operators around the gated delta rule cost: the short causal convolution,
the selective state space scan (prompts and single tokens) and the RMS norm with the
residual's addition and an 8-bit output. ``run`` computes them in plain torch, or through
this package where ``own`` is true."""
import importlib
import math
import random

import torch

own = False
_PKG = "gated_delta_rule_64_amd"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_FP8_MAX = 448.0      # the largest e4m3 value
_TINY = 2.0 ** -110   # an 8-bit row's largest value counts as at least this


# ---------------------------------------------------------------------------- the cases
def listed():
    return [
        # the convolution of q, k and v together ahead of the long-context KDA layer
        # (H = 16, HV = 32, K = V = 128: 2*16*128 + 32*128 channels), a whole prompt
        dict(name="conv prompt", op="conv", dir="fwd", dtype="bf16", B=1, T=8192, D=8192, W=4, silu=True, state=False),
        # the same for H = HV = 16 over a packed batch of ragged prompts that go on from a cache
        dict(name="conv packed", op="conv", dir="fwd", dtype="bf16", slots=64, lo=1, hi=1024, empty=4, lens=3, D=6144,
             W=4, silu=True, state=True),
        # a training step's gradient of it
        dict(name="conv backward", op="conv", dir="bwd", dtype="bf16", B=2, T=4096, D=6144, W=4, silu=True, state=False),
        # one token of each running sequence
        dict(name="conv step", op="conv", dir="fwd", dtype="bf16", B=256, T=1, D=8192, W=4, silu=True, state=True),
        # the long-context layer's sizes, one prompt
        dict(name="scan prompt", op="scan", dir="chunk", dtype="bf16", B=1, T=8192, H=16, HV=32, K=128, V=128, state=False),
        # a long document, one b / c group shared by all heads
        dict(name="scan long", op="scan", dir="chunk", dtype="bf16", B=1, T=32768, H=1, HV=64, K=128, V=64, state=True),
        # a packed batch of ragged prompts that go on from cached states
        dict(name="scan packed", op="scan", dir="chunk", dtype="bf16", slots=64, lo=1, hi=1024, empty=4, lens=5, H=16,
             HV=16, K=128, V=128, state=True),
        # short odd prompts in full precision, where latency counts
        dict(name="scan short", op="scan", dir="chunk", dtype="f32", B=3, T=77, H=2, HV=4, K=64, V=64, state=True),
        # one token of each of many running sequences
        dict(name="scan step", op="scan", dir="step", dtype="bf16", B=1024, T=1, H=16, HV=32, K=128, V=128, state=True),
        # a prompt's rows at the entry of a layer whose projections take 8-bit inputs
        dict(name="norm 8-bit", op="norm", dir="quant", dtype="bf16", rows=8192, D=4096, group=0, residual=True),
        # the rows of a few running sequences, scales for 128 columns each
        dict(name="norm 8-bit few rows", op="norm", dir="quant", dtype="bf16", rows=16, D=4096, group=128, residual=True),
        # a training step's gradient of the norm, with the residual stream's
        dict(name="norm backward", op="norm", dir="bwd", dtype="bf16", rows=8192, D=4096, residual=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Sizes over the ranges above: rows of any length, channels in steps of 8 and odd ones, W of 2 to 4,
    every head layout of the scan, both types, dense and packed, with and without cached states."""
    op = rng.choice(("conv", "conv", "scan", "scan", "scan", "norm", "norm"))
    c = {"op": op, "dtype": rng.choice(("bf16", "bf16", "bf16", "f32"))}
    if op == "norm":
        c["dir"] = rng.choice(("quant", "quant", "fwd", "bwd"))
        c["rows"] = _log(rng, 1, 8192)
        c["D"] = _log(rng, 64, 4096) if rng.random() < 0.3 else 128 * _log(rng, 1, 32)
        if c["dir"] == "quant":
            c["group"] = 128 if c["D"] % 128 == 0 and rng.random() < 0.5 else 0
        c["residual"] = rng.random() < 0.7
        return c
    if op == "scan":
        c["K"], c["V"] = rng.choice((64, 128)), rng.choice((64, 128))
        c["H"] = rng.choice((1, 2, 4, 8))
        c["HV"] = c["H"] * rng.choice((1, 2, 3, 4))
        c["state"] = rng.random() < 0.5
        if rng.random() < 0.35:
            c.update(dir="step", B=_log(rng, 1, 1024), T=1, state=True)
            return c
        c["dir"] = "chunk"
        most = (32768 if c["dtype"] == "bf16" else 4096) * 16 // max(16, c["HV"])
    else:
        c["dir"] = rng.choice(("fwd", "fwd", "bwd"))
        c["D"] = _log(rng, 64, 8192) if rng.random() < 0.2 else 8 * _log(rng, 8, 1024)
        c["W"], c["silu"], c["state"] = rng.choice((2, 3, 4, 4)), rng.random() < 0.8, rng.random() < 0.5
        most = 8192 * 6144 // max(6144, c["D"])
    if rng.random() < 0.4:
        slots = rng.randint(2, 48)
        hi = max(2, _log(rng, 2, max(2, most // slots)))
        c.update(slots=slots, lo=1, hi=hi, empty=rng.randint(0, min(3, slots - 1)), lens=rng.randint(0, 1 << 20))
    else:
        c["B"] = rng.choice((1, 1, 2, 3))
        c["T"] = _log(rng, 1, most // c["B"])
    return c


def _lengths(case):
    """Each sequence's length."""
    if "slots" not in case:
        return [case["T"]] * case["B"]
    r = random.Random(case["lens"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["slots"])]
    for i in r.sample(range(case["slots"]), case["empty"]):
        lens[i] = 0
    return lens


def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] == "norm":
        n = case["rows"] * case["D"]
        if case["dir"] == "bwd":
            moved = n * e * (4 if case["residual"] else 3) + case["D"] * (e + 4) + case["rows"] * 4
            return {"bytes": moved, "flops": 10 * n}
        out = n * (1 if case["dir"] == "quant" else e) + n * e * (3 if case["residual"] else 1)
        scales = 4 * case["rows"] * (1 if case["dir"] == "fwd" or not case["group"] else case["D"] // case["group"])
        return {"bytes": out + scales + case["D"] * e, "flops": 6 * n}
    lens = _lengths(case)
    rows, N = sum(lens), len(lens)
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        states = N * D * (W - 1) * e * ((2 if case["dir"] == "fwd" else 2) if case["state"] else 1)
        n = rows * D
        if case["dir"] == "fwd":
            return {"bytes": 2 * n * e + states + D * (W + 1) * e, "flops": n * (2 * W + 5)}
        return {"bytes": 3 * n * e + states + D * (W + 1) * (e + 4), "flops": n * (6 * W + 12)}
    H, HV, K, V = (case[k] for k in ("H", "HV", "K", "V"))
    moved = rows * (2 * HV * V * e + 2 * H * K * e + HV * e) + N * HV * K * V * 4 * (2 if case["state"] else 1)
    # the state's update and its read-out for each token and head
    return {"bytes": moved, "flops": rows * HV * (4 * K * V + 2 * V)}


# ------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo

    s = {"case": case}
    if case["op"] == "norm":
        rows, D = case["rows"], case["D"]
        s["w"] = (1.0 + 0.1 * randn(D)).to(dt)
        if case["dir"] == "bwd":
            s["h"] = (2.0 * randn(rows, D)).to(dt)
            s["dy"] = randn(rows, D).to(dt)
            s["rstd"] = (s["h"].double().square().mean(-1) + 1e-6).rsqrt().float()
            s["dh"] = randn(rows, D).to(dt) if case["residual"] else None
        else:
            s["x"] = randn(rows, D).to(dt)
            s["residual"] = (2.0 * randn(rows, D)).to(dt) if case["residual"] else None
        return s
    lens = _lengths(case)
    N = len(lens)
    s["max_len"], s["rows"] = max(lens), sum(lens)
    s["cu"] = None
    B, T = (1, sum(lens)) if "slots" in case else (case["B"], case["T"])
    if "slots" in case:
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n)
        s["cu"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        s["x"] = randn(B, T, D).to(dt)
        s["w"] = uniform(-0.5, 0.5, D, W).to(dt)
        s["bias"] = uniform(-0.5, 0.5, D).to(dt)
        s["state"] = randn(N, W - 1, D).to(dt) if case["state"] else None
        if case["dir"] == "bwd":
            s["dy"] = randn(B, T, D).to(dt)
            s["dstate"] = randn(N, W - 1, D).to(dt) if case["state"] else None
        return s
    H, HV, K, V = (case[k] for k in ("H", "HV", "K", "V"))
    silu = torch.nn.functional.silu
    s["x"], s["b"], s["c"] = silu(randn(B, T, HV, V)).to(dt), silu(randn(B, T, H, K)).to(dt), silu(randn(B, T, H, K)).to(dt)
    s["dt"] = (0.5 * randn(B, T, HV)).to(dt)
    s["A_log"] = uniform(1.0, 16.0, HV).log()
    step = uniform(math.log(1e-3), math.log(1e-1), HV).exp()   # the usual start: steps of 1e-3 to 1e-1
    s["dt_bias"] = step + (-torch.expm1(-step)).log()
    s["D"] = 1.0 + 0.1 * randn(HV)
    s["state"] = randn(N, HV, K, V) if case["state"] else None
    return s


# ------------------------------------------------------------------- through the package
def _own(s):
    kda = importlib.import_module(_PKG)
    case = s["case"]
    if case["op"] == "norm":
        if case["dir"] == "bwd":
            return kda.kda_rmsnorm_bwd(s["dy"], s["h"], s["w"], s["rstd"], s["dh"])
        if case["dir"] == "quant":
            return kda.kda_rmsnorm_quant_fwd(s["x"], s["w"], s["residual"], eps=1e-6, group=case["group"])
        return kda.kda_rmsnorm_fwd(s["x"], s["w"], s["residual"], eps=1e-6, output_rstd=True)
    if case["op"] == "conv":
        act = "silu" if case["silu"] else None
        if case["dir"] == "bwd":
            return kda.kda_conv_bwd(s["dy"], s["x"], s["w"], s["bias"], s["state"], s["cu"], s["dstate"], activation=act)
        return kda.kda_conv_fwd(s["x"], s["w"], s["bias"], s["state"], s["cu"], output_final_state=True, activation=act)
    f = kda.kda_ssm_recurrent_fwd if case["dir"] == "step" else kda.kda_ssm_chunk_fwd
    return f(s["x"], s["dt"], s["A_log"], s["b"], s["c"], s["D"], s["dt_bias"], s["state"], s["cu"],
             output_final_state=True, dt_softplus=True)


# ----------------------------------------------------------------------- the plain forms
def _packed_places(s, W1):
    """For a packed batch: each row's sequence and place in it, and for tap i (i rows back) its row in
    [state rows; token rows], as one index over the rows of both laid end to end."""
    cu = s["cu"].long()
    t = torch.arange(s["rows"], device=cu.device)
    n = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = t - cu[n]
    back = torch.arange(W1, -1, -1, device=cu.device)[None]
    inside = pos[:, None] >= back
    first = (cu.numel() - 1) * W1
    return torch.where(inside, first + t[:, None] - back, n[:, None] * W1 + W1 + pos[:, None] - back)


def _conv_taps(s):
    """fp32 [sequences' rows..., W, D]: each row with the W - 1 rows before it."""
    case, x = s["case"], s["x"].float()
    W1, D = case["W"] - 1, case["D"]
    N = s["cu"].numel() - 1 if s["cu"] is not None else case["B"]
    state = s["state"].float() if s["state"] is not None else x.new_zeros(N, W1, D)
    if s["cu"] is None:
        ext = torch.cat([state, x], 1)
        return ext.unfold(1, W1 + 1, 1).transpose(2, 3), ext, None
    ext = torch.cat([state.reshape(N * W1, D), x[0]], 0)
    at = _packed_places(s, W1)
    return ext[at][None], ext, at


def _last_rows(s, ext):
    """Where the last W - 1 rows of every sequence (its state's rows counted first) are in ext."""
    W1 = s["case"]["W"] - 1
    cu = s["cu"].long()
    N = cu.numel() - 1
    lens = cu[1:] - cu[:-1]
    back = torch.arange(W1, 0, -1, device=cu.device)[None]
    pos = lens[:, None] - back
    return torch.where(pos >= 0, N * W1 + cu[:-1, None] + pos, torch.arange(N, device=cu.device)[:, None] * W1 + W1 + pos)


def _plain_conv(s):
    case = s["case"]
    dt = s["x"].dtype
    W1 = case["W"] - 1
    taps, ext, _ = _conv_taps(s)
    w = s["w"].float().t()
    y = (taps * w).sum(-2) + s["bias"].float()
    if case["silu"]:
        y = y / (1.0 + torch.exp(-y))
    last = ext[:, ext.shape[1] - W1:] if s["cu"] is None else ext[_last_rows(s, ext)]
    return y.to(dt), last.to(dt)


def _plain_conv_bwd(s):
    case = s["case"]
    dt = s["x"].dtype
    W, W1 = case["W"], case["W"] - 1
    taps, ext, at = _conv_taps(s)
    w = s["w"].float().t()
    d = s["dy"].float()
    if case["silu"]:
        pre = (taps * w).sum(-2) + s["bias"].float()
        sg = 1.0 / (1.0 + torch.exp(-pre))
        d = d * (sg * (1.0 + pre * (1.0 - sg)))
    # long sums over the rows: in 64 bits
    dw = (d[..., None, :] * taps).sum((0, 1), dtype=torch.float64).t().float()
    db = d.sum((0, 1), dtype=torch.float64).float()
    each = d[..., None, :] * w
    dext = torch.zeros_like(ext)
    if s["cu"] is None:
        T = case["T"]
        parts = [torch.nn.functional.pad(each[:, :, i], (0, 0, i, W1 - i)) for i in range(W)]
        dext = torch.stack(parts).sum(0) if T else dext
        if s["dstate"] is not None:
            dext[:, dext.shape[1] - W1:] += s["dstate"].float()
        dstate, dx = dext[:, :W1], dext[:, W1:]
    else:
        N = s["cu"].numel() - 1
        dext.index_add_(0, at.reshape(-1), each.reshape(-1, case["D"]))
        if s["dstate"] is not None:
            dext.index_add_(0, _last_rows(s, ext).reshape(-1), s["dstate"].float().reshape(-1, case["D"]))
        dstate, dx = dext[: N * W1].view(N, W1, -1), dext[N * W1:][None]
    return dx.to(dt), dw, db, dstate.to(dt) if s["state"] is not None else None


def _padded(s, names, long):
    """The packed rows as [N, max_len, ...], zero behind each sequence's end; dense rows as they are."""
    if s["cu"] is None:
        return [s[n].to(long) for n in names], None
    cu = s["cu"].long()
    t = torch.arange(s["max_len"], device=cu.device)[None]
    there = t < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(there, cu[:-1, None] + t, 0)
    got = []
    for n in names:
        v = s[n][0].to(long)[at]
        got.append(v * there.reshape(there.shape + (1,) * (v.dim() - 2)))
    return got, there


def _steps(s, long):
    """dt' and its log decay [N, L, HV] with nothing behind a sequence's end."""
    (raw,), there = _padded(s, ["dt"], long)
    z = raw + s["dt_bias"].to(long)
    step = torch.clamp_min(z, 0) + torch.log1p(torch.exp(-z.abs()))
    if there is not None:
        step = step * there[..., None]
    return step, -torch.exp(s["A_log"].to(long)) * step, there


def _plain_scan(s):
    case = s["case"]
    H, HV, K, V = (case[k] for k in ("H", "HV", "K", "V"))
    f32, f64 = torch.float32, torch.float64
    step, decay, there = _steps(s, f64)      # angles of a kind: exponents of far rows, in 64 bits
    (x, b, c), _ = _padded(s, ["x", "b", "c"], f32)
    N, L = x.shape[:2]
    Q = min(128, max(1, L))
    NC = -(-L // Q)
    grow = NC * Q - L
    pad = lambda v: torch.nn.functional.pad(v, (0, 0) * (v.dim() - 2) + (0, grow)) if grow else v  # noqa: E731
    cut = lambda v: pad(v).reshape(N, NC, Q, *v.shape[2:]).transpose(2, 3)  # noqa: E731  [N, NC, heads, Q, ...]
    x_, b_, c_ = cut(x), cut(b), cut(c)
    step_, cum = cut(step).float(), cut(decay).cumsum(-1)                     # [N, NC, HV, Q]
    R = HV // H
    rep = lambda v: v.repeat_interleave(R, 2) if R > 1 else v  # noqa: E731
    keep = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    gap = (cum[..., :, None] - cum[..., None, :]).masked_fill(~keep, -math.inf).float()
    m = rep(c_ @ b_.transpose(-1, -2)) * torch.exp(gap) * step_[..., None, :]
    y = m @ x_
    tail = (cum[..., -1:] - cum).float()
    part = (rep(b_) * (torch.exp(tail) * step_)[..., None]).transpose(-1, -2) @ x_   # [N, NC, HV, K, V]
    h0 = s["state"] if s["state"] is not None else x.new_zeros(N, HV, K, V)
    ends = cum[..., -1].cumsum(1)                                                    # [N, NC, HV]
    ends = torch.cat([torch.zeros_like(ends[:, :1]), ends], 1).transpose(1, 2)       # before chunk c; [N, HV, NC + 1]
    keep = torch.ones(NC + 1, NC + 1, dtype=torch.bool, device=x.device).tril()
    far = torch.exp((ends[..., :, None] - ends[..., None, :]).masked_fill(~keep, -math.inf).float())
    parts = torch.cat([h0[:, None], part], 1).transpose(1, 2).reshape(N, HV, NC + 1, K * V)
    starts = (far @ parts).view(N, HV, NC + 1, K, V)
    y = y + (rep(c_) * torch.exp(cum.float())[..., None]) @ starts[:, :, :NC].transpose(1, 2)
    y = y.transpose(2, 3).reshape(N, NC * Q, HV, V)[:, :L] + s["D"][:, None] * x
    if there is not None:
        y = y[there][None]
    return y.to(s["x"].dtype), starts[:, :, NC].contiguous()


def _plain_step(s):
    """One token of every sequence."""
    case = s["case"]
    R = case["HV"] // case["H"]
    step, decay, _ = _steps(s, torch.float32)
    x, b, c = s["x"][:, 0].float(), s["b"][:, 0].float(), s["c"][:, 0].float()
    if R > 1:
        b, c = b.repeat_interleave(R, 1), c.repeat_interleave(R, 1)
    S = s["state"] * torch.exp(decay[:, 0])[..., None, None] + b[..., None] * (step[:, 0, :, None] * x)[..., None, :]
    y = (c[..., None] * S).sum(-2) + s["D"][:, None] * x
    return y[:, None].to(s["x"].dtype), S


def _plain_norm(s):
    case = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    r = torch.rsqrt(h.square().mean(-1) + 1e-6)
    y = h * r[:, None] * s["w"].float()
    kept = h.to(s["x"].dtype) if s["residual"] is not None else None
    if case["dir"] == "fwd":
        return y.to(s["x"].dtype), kept, r
    rows, D = y.shape
    g = case["group"] or D
    y = y.view(rows, D // g, g)
    scale = y.abs().amax(-1).clamp_min(_TINY) / _FP8_MAX
    q = (y / scale[..., None]).to(torch.float8_e4m3fn)
    return q.view(rows, D), scale, kept


def _plain_norm_bwd(s):
    dy, h, w, r = s["dy"].float(), s["h"].float(), s["w"].float(), s["rstd"][:, None]
    xhat = h * r
    g = w * dy
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(s["h"].dtype), (dy * xhat).sum(0, dtype=torch.float64).float()


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "norm":
        return _plain_norm_bwd(state) if case["dir"] == "bwd" else _plain_norm(state)
    if case["op"] == "conv":
        return _plain_conv_bwd(state) if case["dir"] == "bwd" else _plain_conv(state)
    return _plain_step(state) if case["dir"] == "step" else _plain_scan(state)


# ------------------------------------------------- the definitions in 64 bits, row by row
def _rows_of(s, lens):
    """(sequence, first row, length) with rows counted over the flattened batch."""
    at, out = 0, []
    for n, ln in enumerate(lens):
        out.append((n, at, ln))
        at += ln
    return out


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        w = s["w"].to(f64)
        if case["dir"] == "bwd":
            h, dy, r = s["h"].to(f64), s["dy"].to(f64), s["rstd"].to(f64)
            D = case["D"]
            dot = torch.mv(dy * h, w)
            dx = dy * w * r[:, None] - h * (dot * r.pow(3) / D)[:, None]
            if s["dh"] is not None:
                dx += s["dh"].to(f64)
            return dx, torch.mv((dy * h).t(), r)
        h = s["x"].to(f64)
        if s["residual"] is not None:
            h = h + s["residual"].to(f64)
        r = 1.0 / torch.sqrt((h * h).sum(-1) / case["D"] + 1e-6)
        y = h * torch.outer(r, w)
        kept = h if s["residual"] is not None else None
        if case["dir"] == "fwd":
            return y, kept, r
        g = case["group"] or case["D"]
        top = torch.stack([p.abs().max(-1).values for p in y.split(g, -1)], -1)
        scale = torch.clamp(top, min=_TINY) / _FP8_MAX
        return y / scale.repeat_interleave(g, -1), scale, kept
    lens = _lengths(case)
    if case["op"] == "conv":
        W, W1, D = case["W"], case["W"] - 1, case["D"]
        x = s["x"].reshape(-1, D)
        w, bias = s["w"].to(f64), s["bias"].to(f64)
        ys, lasts, dxs, dstates = [], [], [], []
        dw, db = torch.zeros(D, W, dtype=f64, device="cuda"), torch.zeros(D, dtype=f64, device="cuda")
        for n, at, ln in _rows_of(s, lens):
            before = s["state"][n].to(f64) if s["state"] is not None else x.new_zeros(W1, D, dtype=f64)
            seq = torch.cat([before, x[at:at + ln].to(f64)])
            pre = bias.expand(ln, D).clone()
            for i in range(W):
                pre += seq[i:i + ln] * w[:, i]
            sg = torch.sigmoid(pre)
            if case["dir"] == "fwd":
                ys.append(pre * sg if case["silu"] else pre)
                lasts.append(seq[ln:])
                continue
            d = s["dy"].reshape(-1, D)[at:at + ln].to(f64)
            if case["silu"]:
                d = d * (sg + pre * sg * (1.0 - sg))
            grad = torch.zeros_like(seq)
            for i in range(W):
                grad[i:i + ln] += d * w[:, i]
                dw[:, i] += (d * seq[i:i + ln]).sum(0)
            db += d.sum(0)
            if s["dstate"] is not None:
                grad[ln:] += s["dstate"][n].to(f64)
            dxs.append(grad[W1:])
            dstates.append(grad[:W1])
        if case["dir"] == "fwd":
            return torch.cat(ys).view(s["x"].shape), torch.stack(lasts)
        return torch.cat(dxs).view(s["x"].shape), dw, db, torch.stack(dstates) if s["state"] is not None else None
    # the recurrence, one token of every sequence at a time
    H, HV, K, V = (case[k] for k in ("H", "HV", "K", "V"))
    N, L = len(lens), max(lens)
    z = s["dt"].reshape(-1, HV).to(f64) + s["dt_bias"].to(f64)
    dt = torch.logaddexp(z, torch.zeros_like(z))
    keep = torch.exp(dt * -torch.exp(s["A_log"].to(f64)))
    x, b, c = s["x"].reshape(-1, HV, V), s["b"].reshape(-1, H, K), s["c"].reshape(-1, H, K)
    S = s["state"].to(f64) if s["state"] is not None else torch.zeros(N, HV, K, V, dtype=f64, device="cuda")
    starts = torch.tensor([a for _, a, _ in _rows_of(s, lens)], device="cuda")
    order = sorted(range(N), key=lambda n: -lens[n])
    S = S[torch.tensor(order, device="cuda")]
    starts = starts[torch.tensor(order, device="cuda")]
    head = torch.arange(HV, device="cuda") // (HV // H)
    y = torch.zeros(x.shape[0], HV, V, dtype=f64, device="cuda")
    ranked = [lens[n] for n in order]
    live = N
    for t in range(L):
        while live and ranked[live - 1] <= t:
            live -= 1
        r = starts[:live] + t
        u = x[r].to(f64) * dt[r][..., None]
        Sl = S[:live]
        Sl.mul_(keep[r][..., None, None]).addcmul_(b[r][:, head].to(f64)[..., None], u[..., None, :])
        y[r] = (c[r][:, head].to(f64)[..., None, :] @ Sl)[..., 0, :]
    y += s["D"].to(f64)[:, None] * x.to(f64)
    back = torch.empty(N, dtype=torch.long, device="cuda")
    back[torch.tensor(order, device="cuda")] = torch.arange(N, device="cuda")
    return y.view(s["x"].shape), S[back]
