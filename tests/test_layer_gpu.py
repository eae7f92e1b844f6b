"""Parity of the operators around the mixer with their fp64 oracle on MI355X.

Tolerances are element by element, from the roundings a result goes through: EPS is fp32's
half step (2^-24), OUT[dtype] the half step of the type an output is stored in (bf16 2^-8,
relative to the value). A sum of n products carries at most (n + 1) EPS of the sum of their
magnitudes; the oracle gives that sum beside every value.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_64_amd as kda
from oracle import layer

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 2.0 ** -24
OUT = {BF: 2.0 ** -8, F32: EPS}
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _ready():
    kda.load_library()
    assert torch.cuda.is_available()
    yield


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(name, got, want, bound):
    """|got - want| <= bound everywhere, NaN in want meaning a row nothing writes."""
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    m = ~np.isnan(want)
    assert np.isfinite(got[m]).all(), f"{name}: not finite"
    over = np.abs(got - want)[m] - np.broadcast_to(bound, want.shape)[m]
    assert over.size == 0 or over.max() <= 0, f"{name}: {over.max():.3e} over its bound"


def offsets(lens, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(lens)]), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------ the convolution
def conv_case(seed, dtype, wdtype, W, D, lens=None, B=1, T=0, bias=True, state=True, tail=0, wide=False):
    g = gen(seed)
    if lens is not None:
        T = sum(lens) + tail
    N = len(lens) if lens is not None else B
    x = randn(g, B, T, D + 24, dtype=dtype)[:, :, 16:16 + D] if wide else randn(g, B, T, D, dtype=dtype)
    return dict(x=x, weight=randn(g, D, W, dtype=wdtype, scale=0.5), bias=randn(g, D, dtype=wdtype, scale=0.5) if bias else None,
                initial_state=randn(g, N, W - 1, D, dtype=dtype) if state else None,
                cu_seqlens=offsets(lens) if lens is not None else None)


def conv_oracle(c, silu):
    B, T, D = c["x"].shape
    seqs = layer.spans(B, T, None if c["cu_seqlens"] is None else c["cu_seqlens"].tolist())
    return layer.conv_fwd(f64(c["x"]).reshape(B * T, D), f64(c["weight"]), f64(c["bias"]), f64(c["initial_state"]), seqs, silu), seqs


def act_bound(pre_mag, y, dtype):
    # pre: at most W + 1 = 5 roundings of the terms' magnitude; SiLU's slope is under 1.1; the
    # sigmoid: the exponent's rounding (EPS |pre| ln 2, doubled for the product with log2 e),
    # v_exp_f32, the sum, v_rcp_f32 at 2 EPS each and the product
    return 1.1 * 5 * EPS * pre_mag + np.abs(y) * (2 * pre_mag + 10) * EPS + OUT[dtype] * np.abs(y) * 1.01 + 1e-37


CONV = [
    dict(dtype=BF, wdtype=BF, W=4, D=520, B=2, T=37),
    dict(dtype=BF, wdtype=F32, W=3, D=64, B=3, T=1),
    dict(dtype=F32, wdtype=F32, W=4, D=132, B=1, T=65),
    dict(dtype=F32, wdtype=BF, W=2, D=7, B=2, T=5),
    dict(dtype=BF, wdtype=BF, W=4, D=1, B=1, T=16),
    dict(dtype=BF, wdtype=BF, W=4, D=77, B=1, T=33, bias=False, state=False),
    dict(dtype=BF, wdtype=BF, W=4, D=1032, lens=[1, 0, 2, 3, 4, 0, 17, 33, 16, 1], tail=5),
    dict(dtype=F32, wdtype=F32, W=3, D=36, lens=[0, 0, 40, 1], tail=1, state=False),
    dict(dtype=BF, wdtype=BF, W=2, D=65, lens=[3] * 70, tail=3),
    dict(dtype=BF, wdtype=BF, W=4, D=64, B=2, T=40, wide=True),
    dict(dtype=BF, wdtype=BF, W=4, D=61, B=2, T=18, wide=True),
    dict(dtype=BF, wdtype=BF, W=4, D=16, B=4, T=0),
    dict(dtype=BF, wdtype=BF, W=4, D=16, lens=[0, 0], tail=0),
]


@pytest.mark.parametrize("i", range(len(CONV)))
@pytest.mark.parametrize("silu", [True, False])
def test_conv_forward(i, silu):
    c = conv_case(100 + i, **CONV[i])
    B, T, D = c["x"].shape
    sentinel = torch.full((B, T, D), 7.0, dtype=c["x"].dtype, device=DEV)
    y, final = kda.kda_conv_fwd(**c, output_final_state=True, activation="silu" if silu else None, out=sentinel, debug=True)
    (wy, wf, mag), _ = conv_oracle(c, silu)
    y = y.view(B * T, D)
    near("y", y, wy, act_bound(mag, wy, c["x"].dtype) if silu else 5 * EPS * mag + OUT[c["x"].dtype] * np.abs(wy) * 1.01)
    assert (f64(y)[np.isnan(wy)] == 7.0).all(), "rows outside every sequence stay as they were"
    assert np.array_equal(f64(final), wf), "the final state is the rows themselves"


@pytest.mark.parametrize("i", range(len(CONV)))
@pytest.mark.parametrize("silu", [True, False])
def test_conv_backward(i, silu):
    c = conv_case(200 + i, **CONV[i])
    B, T, D = c["x"].shape
    W, dtype = c["weight"].shape[1], c["x"].dtype
    g = gen(300 + i)
    N = c["cu_seqlens"].numel() - 1 if c["cu_seqlens"] is not None else B
    dy = randn(g, B, T, D, dtype=dtype)
    df = randn(g, N, W - 1, D, dtype=dtype) if i % 2 else None
    dx, dw, db, dh = kda.kda_conv_bwd(dy, **c, dfinal_state=df, activation="silu" if silu else None, debug=True)
    seqs = layer.spans(B, T, None if c["cu_seqlens"] is None else c["cu_seqlens"].tolist())
    *want, mag = layer.conv_bwd(f64(dy).reshape(B * T, D), f64(c["x"]).reshape(B * T, D), f64(c["weight"]), f64(c["bias"]),
                                f64(c["initial_state"]), f64(df), seqs, silu)
    # dpre: the pre-activation's 5 roundings of its magnitude A (at most `top`) through slopes
    # under 1.1, the sigmoid's (2 A + 10) and a few products; then sums of rows
    rows = sum(ln for _, ln in seqs)
    top = np.nanmax(conv_oracle(c, silu)[0][2]) if rows else 0.0
    each = (10 * top + 40) * EPS if silu else 2 * EPS
    out = OUT[dtype] * 1.01
    # a term's error is relative to |dy| where silu's slope is small: bound by |dy| itself
    dmag = np.abs(f64(dy).reshape(B * T, D)) if silu else 0.0
    slack = each * (np.max(dmag) if rows and silu else 0.0) * 4 * np.abs(f64(c["weight"])).sum(1)
    near("dx", dx.view(B * T, D)[torch.tensor(~np.isnan(want[0][:, 0]), device=DEV)] if rows else dx.view(B * T, D)[:0],
         want[0][~np.isnan(want[0][:, 0])], ((each + 6 * EPS) * mag[0] + out * np.abs(np.nan_to_num(want[0])) + slack)[~np.isnan(want[0][:, 0])])
    if c["cu_seqlens"] is not None and rows < T:
        assert not f64(dx.view(B * T, D))[np.isnan(want[0])].any(), "rows outside every sequence are zero"
    big = np.max(np.abs(f64(c["x"]))) if c["x"].numel() else 0.0
    if c["initial_state"] is not None and c["initial_state"].numel():
        big = max(big, np.max(np.abs(f64(c["initial_state"]))))
    sum_slack = each * (np.max(dmag) if rows and silu else 0.0) * rows
    near("dw", dw, want[1], (each + (rows + 2) * EPS) * mag[1] + sum_slack * big)
    if c["bias"] is not None:
        near("db", db, want[2], (each + (rows + 2) * EPS) * mag[2] + sum_slack)
    else:
        assert db is None
    if c["initial_state"] is not None:
        near("dinitial", dh, want[3], (each + 6 * EPS) * mag[3] + out * np.abs(want[3]) + slack)
    else:
        assert dh is None


def test_conv_step_by_step_is_the_prompt_bitwise():
    c = conv_case(1, BF, BF, 4, 264, B=3, T=21)
    y, final = kda.kda_conv_fwd(**c, output_final_state=True)
    x, state, rows = c["x"], c["initial_state"].clone(), []
    for t in range(x.shape[1]):   # in place: final_state is initial_state
        o, s = kda.kda_conv_fwd(x[:, t:t + 1], c["weight"], c["bias"], state, output_final_state=True, final_state=state)
        assert s is state
        rows.append(o)
    assert torch.equal(torch.cat(rows, 1), y) and torch.equal(state, final)


def test_conv_in_place_state_of_packed_prompts():
    c = conv_case(2, BF, BF, 4, 136, lens=[1, 40, 0, 2, 3, 64])
    y, final = kda.kda_conv_fwd(**c, output_final_state=True)
    state = c.pop("initial_state").clone()
    y2, s = kda.kda_conv_fwd(**c, initial_state=state, output_final_state=True, final_state=state)
    assert torch.equal(y, y2) and torch.equal(final, s)


def test_outputs_that_are_inputs_are_refused():
    c = conv_case(9, BF, BF, 4, 64, B=2, T=9)
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(**c, out=c["x"])
    s = ssm_case(9, H=1, HV=2, T=9)
    for f in (kda.kda_ssm_chunk_fwd, kda.kda_ssm_recurrent_fwd):
        with pytest.raises(ValueError):
            f(**s, out=s["x"])


def test_conv_packed_is_the_dense_runs():
    lens = [5, 33, 0, 64]
    c = conv_case(3, BF, BF, 4, 96, lens=lens)
    y, final = kda.kda_conv_fwd(**c, output_final_state=True)
    at = 0
    for n, ln in enumerate(lens):
        o, f = kda.kda_conv_fwd(c["x"][:, at:at + ln], c["weight"], c["bias"], c["initial_state"][n:n + 1], output_final_state=True)
        assert torch.equal(o, y[:, at:at + ln]) and torch.equal(f, final[n:n + 1])
        at += ln


@pytest.mark.parametrize("cu", [[1, 5, 9], [0, 7, 3], [0, 5, 900], [0, -4, 9]])
def test_conv_broken_offsets_are_flagged_and_safe(cu):
    g = gen(4)
    x, w = randn(g, 1, 20, 64, dtype=BF), randn(g, 64, 4, dtype=BF)
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    with pytest.raises(kda.KdaDeviceCheckError):
        kda.kda_conv_fwd(x, w, cu_seqlens=cu, output_final_state=True, debug=True)
    with pytest.raises(kda.KdaDeviceCheckError):
        kda.kda_conv_bwd(x, x, w, cu_seqlens=cu, debug=True)


def test_conv_other_sequences_nan_stays_there():
    c = conv_case(5, BF, BF, 4, 64, lens=[7, 9, 30])
    ref, _ = kda.kda_conv_fwd(**c)
    c["x"][0, 7:16] = float("nan")
    c["initial_state"][1] = float("inf")
    y, _ = kda.kda_conv_fwd(**c)
    assert torch.equal(y[0, :7], ref[0, :7]) and torch.equal(y[0, 16:], ref[0, 16:])
    # and a NaN W rows back is out of reach
    x = randn(gen(6), 1, 12, 64, dtype=BF)
    x[0, 3] = float("nan")
    for W in (2, 3, 4):
        y, _ = kda.kda_conv_fwd(x, randn(gen(7), 64, W, dtype=BF))
        bad = torch.isnan(y).any(-1)[0].nonzero().flatten().tolist()
        assert bad == list(range(3, 3 + W))


def test_rows_beyond_32_bit_offsets():
    """Rows 2^20 elements apart: the last ones lie past 2^32 elements."""
    T, step = 4200, 1 << 20
    big = torch.empty(T * step, dtype=BF, device=DEV)
    g = gen(8)
    x = big.as_strided((1, T, 64), (T * step, step, 1), 0)
    x.copy_(randn(g, 1, T, 64, dtype=BF))
    near_x = x.contiguous()
    w = randn(g, 64, 4, dtype=BF)
    assert torch.equal(kda.kda_conv_fwd(x, w)[0], kda.kda_conv_fwd(near_x, w)[0])
    dy = randn(g, 1, T, 64, dtype=BF)
    for a, b in zip(kda.kda_conv_bwd(dy, x, w)[:2], kda.kda_conv_bwd(dy, near_x, w)[:2]):
        assert torch.equal(a, b)
    n = torch.ones(64, dtype=BF, device=DEV)
    assert torch.equal(kda.kda_rmsnorm_fwd(x[0], n)[0], kda.kda_rmsnorm_fwd(near_x[0], n)[0])
    b, c = randn(g, 1, T, 1, 64, dtype=BF), randn(g, 1, T, 1, 64, dtype=BF)
    dt, A = randn(g, 1, T, 1), torch.zeros(1, device=DEV)
    far = (x.view(1, T, 1, 64) if x.is_contiguous() else x.unflatten(-1, (1, 64)))
    for f in (kda.kda_ssm_chunk_fwd, kda.kda_ssm_recurrent_fwd):
        p = f(far, dt, A, b, c, output_final_state=True, dt_softplus=True)
        q = f(near_x.view(1, T, 1, 64), dt, A, b, c, output_final_state=True, dt_softplus=True)
        assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])


# ------------------------------------------------------------------------------ the scan
def ssm_case(seed, dtype=BF, H=1, HV=2, K=64, V=64, lens=None, B=1, T=0, state=True, D=True, bias=True, softplus=True,
             tail=0, dt_dtype=None, a_log=None, wide=False, dt_scale=1.0):
    g = gen(seed)
    if lens is not None:
        T = sum(lens) + tail
    N = len(lens) if lens is not None else B
    if wide:   # columns of one wider tensor, as a projection or the convolution leaves them
        all_ = randn(g, B, T, 8 + HV * V + 2 * H * K, dtype=dtype)
        x, b, c = (v.unflatten(-1, s) for v, s in zip(all_[:, :, 8:].split([HV * V, H * K, H * K], -1), ((HV, V), (H, K), (H, K))))
        dt = randn(g, B, T, HV + 5, dtype=dt_dtype or dtype)[:, :, 3:3 + HV]
    else:
        x, b, c = randn(g, B, T, HV, V, dtype=dtype), randn(g, B, T, H, K, dtype=dtype), randn(g, B, T, H, K, dtype=dtype)
        dt = randn(g, B, T, HV, dtype=dt_dtype or dtype, scale=dt_scale)
    if not softplus:
        dt = dt.abs()
    A = torch.rand(HV, generator=g, device=DEV) * 15 + 1
    return dict(x=x, dt=dt, A_log=A.log() if a_log is None else torch.full((HV,), a_log, device=DEV), b=b, c=c,
                D=randn(g, HV) if D else None, dt_bias=randn(g, HV) - 3.0 if bias else None,
                initial_state=randn(g, N, HV, K, V) if state else None,
                cu_seqlens=offsets(lens) if lens is not None else None, dt_softplus=softplus)


def ssm_check(c, fn, chunk):
    B, T, HV, V = c["x"].shape
    H, K = c["b"].shape[2:]
    dtype = c["x"].dtype
    sentinel = torch.full((B, T, HV, V), 7.0, dtype=dtype, device=DEV)
    y, final = fn(**c, output_final_state=True, out=sentinel, debug=True)
    seqs = layer.spans(B, T, None if c["cu_seqlens"] is None else c["cu_seqlens"].tolist())
    r = lambda t, *s: f64(t).reshape(B * T, *s)  # noqa: E731
    wy, wf, my, mf = layer.ssm(r(c["x"], HV, V), r(c["dt"], HV), f64(c["A_log"]), r(c["b"], H, K), r(c["c"], H, K), f64(c["D"]),
                               f64(c["dt_bias"]), f64(c["initial_state"]), seqs, c["dt_softplus"])
    # fp32 path: an element is a sum over at most T tokens and K rows of products whose
    # weights 2^E dt' carry the exponent's rounding (|E| up to 150 before it is 0: dt' and the
    # exp of A_log are within 4 EPS, so 150 * 8 EPS), the exponential's 2 EPS and a rounding a
    # token and chunk
    longest = max([ln for _, ln in seqs] + [0])
    steps = (longest + K + 1400) * EPS
    # the chunked bf16 path rounds M and the state to bf16 for the matrix cores (one half
    # step of each term), and the output once
    rel = steps + (OUT[BF] * 1.01 if chunk and dtype == BF else 0.0)
    y = y.view(B * T, HV, V)
    near("y", y, wy, rel * my + OUT[dtype] * 1.01 * np.abs(np.nan_to_num(wy)) * (1 + rel) + 1e-35)
    assert (f64(y)[np.isnan(wy)] == 7.0).all(), "rows outside every sequence stay as they were"
    near("final", final, wf, steps * mf + 1e-35)
    for n, (_, ln) in enumerate(seqs):
        if ln == 0:
            same = c["initial_state"][n] if c["initial_state"] is not None else torch.zeros_like(final[n])
            assert torch.equal(final[n], same)
    return y, final


SSM = [
    dict(H=1, HV=2, T=1, B=2), dict(H=2, HV=2, T=2, K=128), dict(H=1, HV=3, T=63, V=128, K=128),
    dict(H=2, HV=4, T=64, K=128, V=64, B=2), dict(H=1, HV=4, T=65, K=128, V=128), dict(H=2, HV=6, T=130, V=192),
    dict(H=4, HV=4, T=300, K=128, V=128), dict(H=1, HV=1, T=1030, K=128, V=64), dict(H=1, HV=2, T=700, B=3, wide=True),
    dict(H=1, HV=2, T=0, B=3), dict(H=2, HV=4, lens=[1, 0, 64, 65, 127, 0, 200, 3], K=128, V=128, tail=9),
    dict(H=1, HV=2, lens=[0, 0, 0]), dict(H=1, HV=2, lens=[600, 1, 5], state=False, tail=1), dict(H=1, HV=2, T=100, D=False, bias=False),
    dict(H=1, HV=2, T=100, softplus=False, bias=False, dt_dtype=F32), dict(H=1, HV=2, T=200, a_log=7.0, K=128),
    dict(H=1, HV=2, T=200, a_log=90.0), dict(H=1, HV=2, T=400, a_log=-20.0, V=128), dict(H=1, HV=2, T=130, dt_scale=30.0, bias=False),
    dict(H=2, HV=4, lens=[70, 0, 10], wide=True, K=128, V=128, tail=2), dict(H=3, HV=9, T=90, K=64, V=64),
    dict(H=1, HV=1, lens=[2500, 0, 1300], K=64, V=64, tail=4),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(SSM)))
def test_scan_of_prompts(i, dtype):
    ssm_check(ssm_case(400 + i, dtype, **SSM[i]), kda.kda_ssm_chunk_fwd, True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(SSM)))
def test_scan_token_by_token(i, dtype):
    ssm_check(ssm_case(500 + i, dtype, **SSM[i]), kda.kda_ssm_recurrent_fwd, False)


@pytest.mark.parametrize("fn", [kda.kda_ssm_chunk_fwd, kda.kda_ssm_recurrent_fwd])
def test_scan_states(fn):
    """No state is zeros, in place is out of place, and a prompt cut at a chunk goes on
    where it stopped: bitwise."""
    c = ssm_case(1, H=2, HV=4, K=128, V=128, T=200, B=2, state=False)
    y, f = fn(**c, output_final_state=True)
    zero = torch.zeros_like(f)
    y2, f2 = fn(**{**c, "initial_state": zero}, output_final_state=True, final_state=zero)
    assert f2 is zero and torch.equal(y, y2) and torch.equal(f, f2)
    assert fn(**c)[1] is None

    def cut(a, b):
        return {k: v[:, a:b].contiguous() if k in ("x", "dt", "b", "c") else v for k, v in c.items()}
    p, s = fn(**cut(0, 128), output_final_state=True)
    q, s = fn(**{**cut(128, 200), "initial_state": s}, output_final_state=True, final_state=s)
    assert torch.equal(torch.cat([p, q], 1), y) and torch.equal(s, f)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [None, [1500, 0, 64, 700]])
def test_scan_of_long_prompts_in_place(lens, dtype):
    """Prompts long enough to be cut into segments, their states replaced where they are."""
    c = ssm_case(6, dtype, H=1, HV=2, K=64, V=128, T=1500, lens=lens)
    y, f = ssm_check(c, kda.kda_ssm_chunk_fwd, True)
    state = c.pop("initial_state").clone()
    y2, f2 = kda.kda_ssm_chunk_fwd(**c, initial_state=state, output_final_state=True, final_state=state)
    assert f2 is state and torch.equal(f, f2)
    rows = sum(lens) if lens else 1500
    assert torch.equal(y[:rows], y2.view(-1, 2, 128)[:rows])


@pytest.mark.parametrize("fn", [kda.kda_ssm_chunk_fwd, kda.kda_ssm_recurrent_fwd])
def test_scan_is_causal_and_sequences_are_apart(fn):
    lens = [70, 130, 64]
    c = ssm_case(2, H=1, HV=2, K=64, V=64, lens=lens)
    y, f = fn(**c, output_final_state=True)
    d = {k: v.clone() if torch.is_tensor(v) else v for k, v in c.items()}
    for k in ("x", "b", "c", "dt"):
        d[k][0, 70:200] = float("nan")
    d["initial_state"][1] = float("inf")
    y2, f2 = fn(**d, output_final_state=True)
    for a, b in ((0, 70), (200, 264)):
        assert torch.equal(y[0, a:b], y2[0, a:b])
    assert torch.equal(f[0], f2[0]) and torch.equal(f[2], f2[2])
    # a token changes nothing before it
    d = {k: v.clone() if torch.is_tensor(v) else v for k, v in c.items()}
    for k in ("x", "b", "c", "dt"):
        d[k][0, 100] += 1.0
    y3, _ = fn(**d)
    assert torch.equal(y[0, :100], y3[0, :100]) and not torch.equal(y[0, 100:], y3[0, 100:])


@pytest.mark.parametrize("cu", [[1, 50, 90], [0, 70, 30], [0, 50, 9000], [0, -40, 90]])
@pytest.mark.parametrize("fn", [kda.kda_ssm_chunk_fwd, kda.kda_ssm_recurrent_fwd])
def test_scan_broken_offsets_are_flagged_and_safe(fn, cu):
    c = ssm_case(3, H=1, HV=2, T=200, state=False)
    c["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    with pytest.raises(kda.KdaDeviceCheckError):
        fn(**c, output_final_state=True, debug=True)


def test_scan_many_sequences_and_long_packed():
    g = np.random.default_rng(5)
    for lens in ([1] * 300, [int(v) for v in g.integers(0, 400, 20)] + [0, 3000]):
        c = ssm_case(4, H=1, HV=2, lens=lens, tail=3)
        ssm_check(c, kda.kda_ssm_chunk_fwd, True)


def test_two_scans_at_once():
    """Calls on two streams with nothing shared, again and again, are the calls by themselves."""
    cases = [ssm_case(60, H=1, HV=4, K=128, V=64, T=3000), ssm_case(61, H=2, HV=4, lens=[700, 0, 1300, 64], K=128, V=128)]
    alone = [kda.kda_ssm_chunk_fwd(**c, output_final_state=True) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(4):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(kda.kda_ssm_chunk_fwd(**c, output_final_state=True))
    torch.cuda.synchronize()
    for i, (y, f) in enumerate(got):
        assert torch.equal(y, alone[i % 2][0]) and torch.equal(f, alone[i % 2][1])


def test_scan_workspace_of_the_callers():
    """A workspace given by the caller, dirty from another problem, changes nothing."""
    c = ssm_case(62, H=1, HV=2, K=64, V=64, T=2000)
    y, f = kda.kda_ssm_chunk_fwd(**c, output_final_state=True)
    need = kda.kda_ssm_chunk_fwd_workspace_bytes(1, 2000, 1, 2, 64, 64, 1, False, BF)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        y2, f2 = kda.kda_ssm_chunk_fwd(**c, output_final_state=True, workspace=ws)
        assert torch.equal(y, y2) and torch.equal(f, f2)
    with pytest.raises(kda.KdaError):
        kda.kda_ssm_chunk_fwd(**c, workspace=ws[:need - 256])


# ------------------------------------------------------------------------------ the norm
NORM = [(1, 1), (3, 3), (5, 64), (7, 96), (4, 128), (9, 200), (2, 256), (3, 500), (6, 512), (5, 1000), (3, 1024), (5, 2048),
        (3, 2056), (2, 4096), (1030, 4096), (2, 5120), (2, 8192), (2, 8191), (1, 20480), (1, 32768), (0, 64), (1100, 40)]


def norm_case(seed, rows, D, dtype, residual=True, wdtype=None):
    g = gen(seed)
    return randn(g, rows, D, dtype=dtype), randn(g, D, dtype=wdtype or dtype), randn(g, rows, D, dtype=dtype) if residual else None


def norm_bound(D, y, dtype):
    # r: (D / 2 + 6) EPS at most (the sum of squares has all signs alike: D roundings over a
    # tree of partial sums, halved by the root), h its addition's rounding, two products
    return np.abs(y) * ((D / 2 + 12) * EPS + OUT[dtype] * 1.01) + 1e-37


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("rows,D", NORM)
def test_norm_forward(rows, D, residual, dtype):
    x, w, res = norm_case(600 + D, rows, D, dtype, residual, BF if D % 3 else F32)
    y, h, r = kda.kda_rmsnorm_fwd(x, w, res, eps=1e-5, output_rstd=True)
    wy, wh, wr = layer.rmsnorm(f64(x), f64(w), f64(res), 1e-5)
    # the rounding of x + residual is relative to the sum, which the norm's own bound holds
    near("y", y, wy, norm_bound(D, wy, dtype))
    near("rstd", r, wr, np.abs(wr) * (D / 2 + 8) * EPS)
    if residual:
        near("h", h, wh, np.abs(wh) * (OUT[dtype] * 1.01 + EPS))
    else:
        assert h is None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,D", [c for c in NORM if c[0]])
def test_norm_in_8_bits(rows, D, group, dtype):
    x, w, res = norm_case(700 + D, rows, D, dtype, D % 2 == 0)
    if group and D % 128:
        with pytest.raises(ValueError):
            kda.kda_rmsnorm_quant_fwd(x, w, res, group=group)
        return
    x[0] = 0
    if res is not None:
        res[0] = 0    # a row of nothing
    q, s, h = kda.kda_rmsnorm_quant_fwd(x, w, res, eps=1e-5, group=group)
    wy, wh, _ = layer.rmsnorm(f64(x), f64(w), f64(res), 1e-5)
    ws = layer.fp8_scales(wy, group or D)
    near("scales", s, ws, ws * (D / 2 + 16) * EPS)
    # a value is rounded to e4m3 by at most half a step: 2^-4 of it, or of 2^-6 below 2^-6
    per = np.repeat(f64(s), group or D, -1)
    got = f64(q.float()) * per
    assert np.isfinite(got).all()
    bound = np.maximum(np.abs(wy), 2.0 ** -6 * per) * (2.0 ** -4) * (1 + 1e-3) + np.abs(wy) * (D / 2 + 20) * EPS
    assert (np.abs(got - wy) <= bound).all()
    # the largest value of each group is 448 itself
    top = np.abs(f64(q.float())).reshape(rows, -1, group or D).max(-1)
    assert (top[1:] == 448).all() and (top[0] == 0).all() and (f64(s)[0] == np.float32(2.0 ** -110) / np.float32(448)).all()
    if res is not None:
        near("h", h, wh, np.abs(wh) * (OUT[dtype] * 1.01 + EPS))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("rows,D", NORM)
def test_norm_backward(rows, D, residual, dtype):
    h, w, dh = norm_case(800 + D, rows, D, dtype, residual, BF if D % 3 else F32)
    dy = randn(gen(9), rows, D, dtype=dtype)
    rstd = (h.double().square().mean(-1) + 1e-6).rsqrt().float()
    dx, dw = kda.kda_rmsnorm_bwd(dy, h, w, rstd, dh)
    wx, ww = layer.rmsnorm_bwd(f64(dy), f64(h), f64(w), f64(rstd), f64(dh))
    r = f64(rstd)[:, None]
    xh, g = np.abs(f64(h) * r), np.abs(f64(dy) * f64(w))
    mean = (g * xh).mean(-1, keepdims=True) if rows else 0.0
    mag = r * (g + xh * mean) + (0 if dh is None else np.abs(f64(dh)))
    near("dx", dx, wx, mag * (D + 12) * EPS + np.abs(wx) * OUT[dtype] * 1.01)
    near("dw", dw, ww, (np.abs(f64(dy)) * xh).sum(0) * (rows + 4) * EPS)


def test_norm_gradient_is_the_difference():
    x, w, res = norm_case(10, 3, 40, F32)
    dy = randn(gen(11), 3, 40)
    dh = randn(gen(12), 3, 40)
    y, h, r = kda.kda_rmsnorm_fwd(x, w, res, eps=1e-3, output_rstd=True)
    dx, dw = kda.kda_rmsnorm_bwd(dy, h, w, r, dh)
    x64, w64, r64, dy64, dh64 = (f64(t) for t in (x, w, res, dy, dh))

    def value():
        y, h, _ = layer.rmsnorm(x64, w64, r64, 1e-3)
        return (y * dy64).sum() + (h * dh64).sum()
    for got, v in ((dx, x64), (dx, r64), (dw, w64)):
        want = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            old, e = v[i], 1e-5
            v[i] = old + e
            up = value()
            v[i] = old - e
            want[i] = (up - value()) / (2 * e)
            v[i] = old
        # differences of 1e-5 are off by about 1e-9 here; the kernel by tens of EPS of the terms
        assert np.abs(f64(got) - want).max() < 1e-4


def test_norm_strides_aliases_and_odd_values():
    g = gen(13)
    wide = randn(g, 2, 9, 300, dtype=BF)
    x, w = wide[:, :, 8:264], randn(g, 256, dtype=BF)
    flat = kda.kda_rmsnorm_fwd(x.contiguous(), w)[0]
    assert torch.equal(kda.kda_rmsnorm_fwd(x, w)[0], flat)
    odd = wide[:, :, 3:259]     # rows not on 16 bytes: one value at a time
    assert torch.allclose(kda.kda_rmsnorm_fwd(odd, w)[0].float(), kda.kda_rmsnorm_fwd(odd.contiguous(), w)[0].float(), rtol=2.0 ** -7)
    with pytest.raises(kda.KdaError):
        kda.kda_rmsnorm_quant_fwd(odd, w, group=128)
    one = randn(g, 96, dtype=BF)     # a single row, without an axis for it
    assert torch.equal(kda.kda_rmsnorm_fwd(one, w[:96])[0], kda.kda_rmsnorm_fwd(one[None], w[:96])[0][0])
    # h into the residual, y into x
    a, res = x.contiguous(), randn(g, 2, 9, 256, dtype=BF)
    y, h, _ = kda.kda_rmsnorm_fwd(a, w, res)
    b, r2 = a.clone(), res.clone()
    y2, h2, _ = kda.kda_rmsnorm_fwd(b, w, r2, out=b, residual_out=r2)
    assert y2 is b and h2 is r2 and torch.equal(y, y2) and torch.equal(h, h2)
    # a row's NaN or infinity stays its own, as NaN codes in 8 bits
    bad = a.clone()
    bad[0, 3, 7] = float("nan")
    bad[1, 2, 0] = float("inf")
    for group in (0, 128):
        q, s, _ = kda.kda_rmsnorm_quant_fwd(bad, w, group=group)
        q0, s0, _ = kda.kda_rmsnorm_quant_fwd(a, w, group=group)
        rows = torch.ones(2, 9, dtype=torch.bool, device=DEV)
        rows[0, 3] = rows[1, 2] = False
        assert torch.equal(q[rows].float(), q0[rows].float()) and torch.equal(s[rows], s0[rows])
        assert torch.isnan(q[0, 3].float()).all() and torch.isnan(q[1, 2, 0].float())


# --------------------------------------------------------------------- all of it together
def _layer_params(seed, D=256, HV=4, H=2, K=64, V=64):
    g = gen(seed)
    C = HV * V + 2 * H * K
    return dict(norm=1 + randn(g, D, dtype=BF, scale=0.1), proj=randn(g, D, C + HV, dtype=BF, scale=D ** -0.5),
                conv=randn(g, C, 4, dtype=BF, scale=0.5), bias=randn(g, C, dtype=BF, scale=0.2),
                A=(torch.rand(HV, generator=g, device=DEV) * 4 + 1).log(), skip=randn(g, HV), dtb=randn(g, HV) - 2,
                sizes=(D, HV, H, K, V, C))


def _layer_run(p, z, conv_state, state, step, cu=None):
    """The projection's rows z -> convolution of x, b, c side by side -> scan, through views
    of the projection's and the convolution's output."""
    D, HV, H, K, V, C = p["sizes"]
    u, conv_state = kda.kda_conv_fwd(z[:, :, :C], p["conv"], p["bias"], conv_state, cu, output_final_state=True)
    x, b, c = u.split([HV * V, H * K, H * K], -1)
    scan = kda.kda_ssm_recurrent_fwd if step else kda.kda_ssm_chunk_fwd
    y, state = scan(x.unflatten(-1, (HV, V)), z[:, :, C:], p["A"], b.unflatten(-1, (H, K)), c.unflatten(-1, (H, K)), p["skip"],
                    p["dtb"], state, cu, output_final_state=True, dt_softplus=True)
    return y, u, conv_state, state


@pytest.mark.parametrize("quant", [False, True])
def test_layer_prompt_then_steps(quant):
    """norm with the residual -> projection -> convolution -> scan: a prompt of 150 and 6 steps
    after it against the prompt of 156. The norm gives every row the same bits whatever rows
    are beside it; the library's product need not (rows of another batch may be summed in
    another order), so it is formed once, and what follows starts from equal rows."""
    p = _layer_params(14)
    g = gen(15)
    D, HV, H, K, V, C = p["sizes"]
    hidden, res = randn(g, 2, 156, 256, dtype=BF), randn(g, 2, 156, 256, dtype=BF)

    def norm(a, b):
        x, r = hidden[:, a:b].contiguous(), res[:, a:b].contiguous()
        if quant:
            q, s, r = kda.kda_rmsnorm_quant_fwd(x, p["norm"], r)
            return (q.float() * s).to(BF), r
        return kda.kda_rmsnorm_fwd(x, p["norm"], r)[:2]
    h, r = norm(0, 156)
    parts = [norm(0, 150)] + [norm(t, t + 1) for t in range(150, 156)]
    assert torch.equal(torch.cat([v[0] for v in parts], 1), h) and torch.equal(torch.cat([v[1] for v in parts], 1), r)
    z = h @ p["proj"]
    whole, u, cs, st = _layer_run(p, z, None, None, False)
    got = [_layer_run(p, z[:, :150].contiguous(), None, None, False)]
    for t in range(150, 156):
        got.append(_layer_run(p, z[:, t:t + 1].contiguous(), *got[-1][2:], True))
    c, s = got[-1][2:]
    assert torch.equal(torch.cat([v[1] for v in got], 1), u) and torch.equal(c, cs)
    got = torch.cat([v[0] for v in got], 1)
    assert torch.equal(got[:, :128], whole[:, :128])
    # from equal rows, each side is within the scan's own bound (ssm_check) of the same value
    rows = lambda v, *sh: f64(v).reshape(312, *sh)  # noqa: E731
    x, b, cc = u.split([HV * V, H * K, H * K], -1)
    wy, wf, my, mf = layer.ssm(rows(x, HV, V), rows(z[:, :, C:], HV), f64(p["A"]), rows(b, H, K), rows(cc, H, K), f64(p["skip"]),
                               f64(p["dtb"]), None, layer.spans(2, 156), True)
    steps = (156 + K + 1400) * EPS
    rel = steps + OUT[BF] * 1.01
    for y, f in ((whole, st), (got, s)):
        near("y", y.reshape(312, HV, V), wy, rel * my + OUT[BF] * 1.01 * np.abs(wy) * (1 + rel))
        near("final", f, wf, steps * mf)


def test_convolution_feeds_the_delta_rule():
    """q, k and v through one convolution into the chunked and the per-token delta rule."""
    g = gen(16)
    B, T, H, HV, K, V = 1, 100, 2, 4, 64, 64
    C = 2 * H * K + HV * V
    z = randn(g, B, T, C, dtype=BF)
    u, _ = kda.kda_conv_fwd(z, randn(g, C, 4, dtype=BF, scale=0.5))
    q, k, v = (t.contiguous() for t in u.split([H * K, H * K, HV * V], -1))
    q, k, v = q.view(B, T, H, K), k.view(B, T, H, K), v.view(B, T, HV, V)
    gate = -torch.rand(B, T, HV, K, generator=g, device=DEV)
    beta = torch.rand(B, T, HV, generator=g, device=DEV).to(BF)
    a, _ = kda.kda_chunk_fwd_ex(q, k, v, gate, beta, use_qk_l2norm_in_kernel=True)
    b, _ = kda.kda_recurrent_fwd_ex(q, k, v, gate, beta, use_qk_l2norm_in_kernel=True)
    assert (a.float() - b.float()).abs().max() <= 2e-2 * b.float().square().mean().sqrt() + 2.0 ** -7 * b.float().abs().max()


def test_other_stream_and_graph_replays():
    """Every operator on a side stream, and captured once and replayed on new inputs in the
    same buffers, with eager work between: bitwise the eager results."""
    p = _layer_params(17)
    g = gen(18)
    hidden, res = randn(g, 1, 200, 256, dtype=BF), randn(g, 1, 200, 256, dtype=BF)
    cu = offsets([64, 0, 100, 36])
    D, HV, H, K, V, C = p["sizes"]
    cs0, st0 = randn(g, 4, 3, C, dtype=BF), randn(g, 4, HV, K, V)
    dy = randn(g, 1, 200, C, dtype=BF)
    rstd = torch.rand(1, 200, generator=g, device=DEV) + 0.5

    def everything():
        # (the library's matrix product stays outside the captured work)
        h, r, rs = kda.kda_rmsnorm_fwd(hidden, p["norm"], res, output_rstd=True)
        q, s, _ = kda.kda_rmsnorm_quant_fwd(hidden, p["norm"], res, group=128)
        u, cs = kda.kda_conv_fwd(z[:, :, :C], p["conv"], p["bias"], cs0, cu, output_final_state=True)
        x, b, c = u.split([HV * V, H * K, H * K], -1)
        args = (x.unflatten(-1, (HV, V)), z[:, :, C:], p["A"], b.unflatten(-1, (H, K)), c.unflatten(-1, (H, K)), p["skip"], p["dtb"], st0, cu)
        y, st = kda.kda_ssm_chunk_fwd(*args, output_final_state=True, dt_softplus=True)
        y1, st1 = kda.kda_ssm_recurrent_fwd(*args, output_final_state=True, dt_softplus=True)
        grads = kda.kda_conv_bwd(dy, z[:, :, :C], p["conv"], p["bias"], cs0, cu)
        gn = kda.kda_rmsnorm_bwd(hidden, res, p["norm"], rstd, None)
        return [h, r, rs, q.float(), s, u, cs, y, st, y1, st1, *grads, *gn]

    z = randn(g, 1, 200, C + HV, dtype=BF)
    want = everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = everything()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = everything()
    for k in range(4):
        hidden.copy_(randn(gen(30 + k), 1, 200, 256, dtype=BF))
        z.copy_(randn(gen(40 + k), 1, 200, C + HV, dtype=BF))
        dy.copy_(randn(gen(50 + k), 1, 200, C, dtype=BF))
        cu.copy_(offsets([[64, 0, 100, 36], [0, 0, 0, 200], [1, 1, 1, 197], [130, 70, 0, 0]][k]))
        graph.replay()
        torch.cuda.synchronize()
        again = everything()
        torch.cuda.synchronize()
        for a, b, n in zip(kept, again, range(99)):
            assert torch.equal(a, b), f"replay {k}, output {n}"
