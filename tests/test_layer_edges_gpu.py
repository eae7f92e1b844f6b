"""Parity of the operators around the mixer where their precision, odd values and sizes are
at stake. Bounds as in test_layer_gpu: EPS is fp32's half step, OUT a stored type's."""
import numpy as np
import pytest
import torch

import gated_delta_rule_64_amd as kda
from oracle import layer
from tests.test_layer_gpu import BF, DEV, EPS, F32, OUT, conv_case, f64, gen, near, offsets, randn, ssm_case

pytestmark = pytest.mark.gpu

SCANS = [kda.kda_ssm_chunk_fwd, kda.kda_ssm_recurrent_fwd]


@pytest.fixture(scope="module", autouse=True)
def _ready():
    kda.load_library()
    assert torch.cuda.is_available()
    yield


def scan_oracle(c):
    B, T, HV, V = c["x"].shape
    H, K = c["b"].shape[2:]
    r = lambda t, *s: f64(t).reshape(B * T, *s)  # noqa: E731
    seqs = layer.spans(B, T, None if c["cu_seqlens"] is None else c["cu_seqlens"].tolist())
    return layer.ssm(r(c["x"], HV, V), r(c["dt"], HV), f64(c["A_log"]), r(c["b"], H, K), r(c["c"], H, K), f64(c["D"]),
                     f64(c["dt_bias"]), f64(c["initial_state"]), seqs, c["dt_softplus"])


# ------------------------------------------------------------------------------ the scan
@pytest.mark.parametrize("H,HV,K,V", [(1, 2, 64, 64), (1, 1, 128, 128), (2, 2, 128, 64), (1, 3, 128, 128), (1, 4, 128, 64)])
def test_scan_operands_keep_16_bits(H, HV, K, V):
    """A first token's product read by every later one, in its chunk (M) and from the state, and
    the read-out's leading bits taken away by the skip: what is left shows the operands' own
    roundings. dt' is 0 after the first token, so nothing decays and nothing else is written."""
    T = 150
    c = ssm_case(1, BF, H, HV, K, V, T=T, state=False, softplus=False, bias=False, dt_dtype=F32, a_log=0.0)
    g = gen(2)
    c["dt"][:, 1:] = 0
    c["dt"][:, 0] = torch.rand(HV, generator=g, device=DEV) + 0.5
    c["b"][:, 0] = 0
    c["b"][:, 0, :, 5] = 1.375
    c["D"] = torch.full((HV,), -1.0, device=DEV)
    # c . b dt' x is one product, and its leading bits are x of the later tokens
    m = c["c"][..., 5].double().repeat_interleave(HV // H, 2) * 1.375 * c["dt"][:, :1].double()
    c["x"][:, 1:] = (m[..., None] * c["x"][:, :1].double()).to(BF)[:, 1:]
    y, _ = kda.kda_ssm_chunk_fwd(**c)
    wy, _, my, _ = scan_oracle(c)
    # a pair of bf16 is off by at most 2^-8 of 2^-8; M, the state and the sums by fp32 steps
    near("y", y.view(T, HV, V), wy, (2.0 ** -16 * 1.01 + 16 * EPS) * my + OUT[BF] * 1.01 * np.abs(wy))


@pytest.mark.parametrize("fn", SCANS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,HV,V,T", [(1, 2, 64, 64), (2, 2, 64, 40), (1, 2, 128, 1000)])
def test_scan_writes_are_fp32_products(H, HV, V, T, dtype, fn):
    """Token t writes row t % K alone and nothing decays (dt' x b summed over a few tokens): a
    state element is a sum of at most T / K + 1 fp32 products."""
    K = 64
    c = ssm_case(3, dtype, H, HV, K, V, T=T, state=False, softplus=False, bias=False, dt_dtype=F32, a_log=-np.inf)
    t = torch.arange(T, device=DEV)
    keep = torch.zeros(T, K, device=DEV, dtype=dtype)
    keep[t, t % K] = 1
    c["b"] *= keep[None, :, None]
    _, final = fn(**c, output_final_state=True)
    _, wf, _, mf = scan_oracle(c)
    # dt' x, its product with b (three parts of it, added one by one, in the chunked form), the sum
    near("final", final, wf, (8 + 2 * (T // K + 1)) * EPS * mf + 1e-37)


@pytest.mark.parametrize("fn", SCANS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_decays_far_along_a_chunk(dtype, fn):
    """Sixteen tokens of 189 log2 units of decay each, then a write, then little decay: the
    differences of the running sums must keep what a sum near 3000 rounded to fp32 (2e-4) loses."""
    c = ssm_case(4, dtype, 1, 2, 64, 64, T=64, softplus=False, bias=False, dt_dtype=F32, a_log=0.0)
    c["dt"][:, :16] = 131.0
    c["dt"][:, 16:] = c["dt"][:, 16:] * 0.01 + 0.001
    c["x"][:, :16] = 0
    c["x"][:, 17:] = 0
    y, final = fn(**c, output_final_state=True)
    wy, wf, my, mf = scan_oracle(c)
    # E < 2 log2 units over the last 47 tokens: the exponent's rounding E EPS, 2 EPS an exponential
    # and a rounding a product, one factor a token in the per-token form
    rel = (16 if fn is kda.kda_ssm_chunk_fwd else 4 * 48 + 16) * EPS
    near("final", final, wf, rel * mf + 1e-37)
    if dtype == F32:
        near("y", y.view(64, 2, 64), wy, (rel + 70 * EPS) * my + 1e-37)


@pytest.mark.parametrize("fn", SCANS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_softplus(dtype, fn):
    """One token of x = b = 1 leaves dt' itself in the state: softplus within 9 half steps from
    where it underflows to where it is its argument."""
    B, HV = 512, 8
    z = torch.cat([torch.linspace(-86, 0, B * HV // 2), torch.linspace(0, 30, B * HV // 2 - 4), torch.tensor([199.9, 200.0, 250.0, 1e30])])
    ones = lambda *s: torch.ones(*s, dtype=dtype, device=DEV)  # noqa: E731
    _, final = fn(ones(B, 1, HV, 64), z.view(B, 1, HV).to(DEV), torch.zeros(HV, device=DEV), ones(B, 1, 1, 64), ones(B, 1, 1, 64),
                  output_final_state=True, dt_softplus=True)
    want = layer.softplus(f64(z)).reshape(B, HV, 1, 1)
    # the bf16 scan takes dt' x in three bf16 parts, under 1, 2^-7 and 2^-15 of it; the matrix cores
    # take a part below the smallest normal number as 0, which loses less than 2^-126 for each
    # of the two that a normal product can have there
    lost = 2 * 2.0 ** -126 if dtype == BF and fn is kda.kda_ssm_chunk_fwd else 0.0
    near("dt'", final, np.broadcast_to(want, final.shape), np.broadcast_to(9 * EPS * want + lost, final.shape))


@pytest.mark.parametrize("fn", SCANS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [50, 1500])
def test_scan_a_nan_decay_is_nan(T, dtype, fn):
    """A head whose A_log is NaN has NaN results, and no other head."""
    c = ssm_case(5, dtype, 1, 4, 64, 64, T=T)
    y, f = fn(**c, output_final_state=True)
    c["A_log"] = c["A_log"].clone()
    c["A_log"][1] = float("nan")
    y2, f2 = fn(**c, output_final_state=True)
    assert torch.isnan(y2[:, :, 1]).all() and torch.isnan(f2[:, 1]).all()
    rest = [0, 2, 3]
    assert torch.equal(y[:, :, rest], y2[:, :, rest]) and torch.equal(f[:, rest], f2[:, rest])


@pytest.mark.parametrize("fn", SCANS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_extreme_decays(dtype, fn):
    """exp(A_log) beyond fp32 with a step of 0 keeps the state, with any other erases it; an
    infinite step erases it too, and A_log of -inf keeps it."""
    T = 70
    c = ssm_case(6, dtype, 1, 4, 64, 64, T=T, softplus=False, bias=False, dt_dtype=F32, D=False)
    c["A_log"] = torch.tensor([90.0, 300.0, -float("inf"), 0.0], device=DEV)
    c["dt"][:, :] = 0
    y, f = fn(**c, output_final_state=True)
    assert torch.equal(f, c["initial_state"])
    c["dt"][:, 66, :2] = 1e-3          # heads 0, 1: everything before token 66 goes
    c["dt"][:, 66, 3] = float("inf")   # head 3: the same, and what it writes is infinite or NaN
    c["b"][:, 66] = 1.0
    y2, f2 = fn(**c, output_final_state=True)
    assert torch.equal(y[:, :66], y2[:, :66])
    want = (c["dt"][:, 66, :2, None] * c["x"][:, 66, :2].float())[:, :, None, :].expand(-1, -1, 64, -1)
    assert (f2[:, :2] - want).abs().max() <= 4 * EPS * want.abs().max()
    assert torch.equal(f2[:, 2], f[:, 2]) and not torch.isfinite(f2[:, 3]).any()


@pytest.mark.parametrize("fn", SCANS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,HV,K,V", [(1, 2, 64, 64), (2, 2, 64, 64), (1, 2, 128, 128)])
def test_scan_odd_values_reach_nothing_before_them(H, HV, K, V, dtype, fn):
    """A NaN or an infinity in any input of a token leaves every earlier output and, in x, every
    other column as they were."""
    T = 200
    c = ssm_case(7, dtype, H, HV, K, V, T=T)
    y, f = fn(**c, output_final_state=True)
    for name in ("x", "b", "c", "dt"):
        for at in (0, 5, 15, 16, 63, 64, 77, 130, 199):
            for bad in (float("nan"), float("inf")):
                d = {**c, name: c[name].clone()}
                if name == "x":
                    d["x"][0, at, 0, 3] = bad
                else:
                    d[name][0, at] = bad
                y2, f2 = fn(**d, output_final_state=True)
                assert torch.equal(y2[:, :at], y[:, :at]), (name, at, bad)
                if name == "c":
                    assert torch.equal(y2[:, at + 1:], y[:, at + 1:]) and torch.equal(f2, f)
                    assert not torch.isfinite(y2[:, at]).any()
                elif name == "x":
                    other = torch.ones(HV, V, dtype=torch.bool, device=DEV)
                    other[0, 3] = False
                    assert torch.equal(y2[0][:, other], y[0][:, other]) and torch.equal(f2[0].transpose(1, 2)[other], f[0].transpose(1, 2)[other])
                    assert not torch.isfinite(y2[0, at, 0, 3]) and not torch.isfinite(f2[0, 0, :, 3]).any()
                elif name == "b" or bad != bad:
                    assert not torch.isfinite(y2[:, at]).any()


def test_scan_more_segments_than_are_sorted():
    """A packed batch of more than 4096 segments, which the second pass takes as they come."""
    lens = [int(v) for v in np.random.default_rng(8).integers(0, 4, 4500)] + [300, 0, 2]
    c = ssm_case(8, BF, 1, 1, 64, 64, lens=lens, tail=3)
    y, f = kda.kda_ssm_chunk_fwd(**c, output_final_state=True, debug=True)
    y2, f2 = kda.kda_ssm_recurrent_fwd(**c, output_final_state=True)
    wy, wf, my, mf = scan_oracle(c)
    steps = (300 + 64 + 1400) * EPS
    for a, b in ((y, f), (y2, f2)):
        near("y", a.view(-1, 1, 64)[:sum(lens)], wy[:sum(lens)], ((steps + OUT[BF]) * my + OUT[BF] * 1.01 * np.abs(wy))[:sum(lens)])
        near("final", b, wf, steps * mf + 1e-35)


# ------------------------------------------------------------------------ the convolution
def test_conv_longest_sequence():
    """The longest sequence there can be, one channel wide: its last rows against the
    convolution of those rows alone."""
    T, W = 2 ** 31 - 1, 4
    x = torch.zeros(1, T, 1, dtype=BF, device=DEV)
    tail = randn(gen(9), 1, 1000, 1, dtype=BF)
    x[:, -1000:] = tail
    w, bias = randn(gen(10), 1, W, dtype=BF), randn(gen(11), 1, dtype=BF)
    y, f = kda.kda_conv_fwd(x, w, bias, output_final_state=True)
    want, wf = kda.kda_conv_fwd(tail, w, bias, output_final_state=True)
    assert torch.equal(y[:, -1000:], want) and torch.equal(f, wf)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    assert torch.equal(kda.kda_conv_fwd(x, w, bias, cu_seqlens=cu, debug=True)[0][:, -1000:], want)
    assert torch.equal(y[:, 5:6].expand(-1, 1000, -1), y[:, T // 2:T // 2 + 1000])
    del y
    dy = torch.zeros(1, T, 1, dtype=BF, device=DEV)
    dy[:, -1000:] = randn(gen(12), 1, 1000, 1, dtype=BF)
    dx, dw, db, _ = kda.kda_conv_bwd(dy, x, w, bias)
    wx, ww, wb, _ = kda.kda_conv_bwd(dy[:, -1000:].contiguous(), tail, w, bias)
    assert torch.equal(dx[:, -1000:], wx) and not dx[:, :1 << 20].any()
    # the same 1000 terms, added in another order
    near("dw", dw, f64(ww), 2 * 1004 * EPS * 1.1 * np.abs(f64(dy[:, -1000:])).sum() * np.abs(f64(tail)).max())


def conv_sums_case(i):
    rng = np.random.default_rng(20 + i)
    return [dict(dtype=F32, wdtype=F32, W=4, D=1024, B=1, T=34000),
            dict(dtype=BF, wdtype=BF, W=3, D=449, lens=[int(v) for v in rng.integers(0, 90, 800)], tail=7),
            dict(dtype=BF, wdtype=F32, W=4, D=1024, lens=[1, 0, 2] * 400 + [9000, 63, 64, 65], tail=1),
            dict(dtype=BF, wdtype=BF, W=2, D=8, B=1, T=70000)][i]


@pytest.mark.parametrize("i", range(4))
def test_conv_backward_of_many_tiles_a_block(i):
    """So many tiles that a block walks several, the last round uneven (and, narrow, one each)."""
    c = conv_case(30 + i, **conv_sums_case(i))
    B, T, D = c["x"].shape
    dy = randn(gen(40 + i), B, T, D, dtype=c["x"].dtype)
    dx, dw, db, dh = kda.kda_conv_bwd(dy, **c, activation=None)
    seqs = layer.spans(B, T, None if c["cu_seqlens"] is None else c["cu_seqlens"].tolist())
    *want, mag = layer.conv_bwd(f64(dy).reshape(T, D), f64(c["x"]).reshape(T, D), f64(c["weight"]), f64(c["bias"]),
                                f64(c["initial_state"]), None, seqs, False)
    out = OUT[c["x"].dtype] * 1.01
    live = ~np.isnan(want[0][:, 0])
    near("dx", dx.view(T, D)[torch.tensor(live, device=DEV)], want[0][live], 6 * EPS * mag[0][live] + out * np.abs(want[0][live]))
    # each tile of 64 rows is summed in fp32, the tiles' sums beyond it
    near("dw", dw, want[1], 70 * EPS * mag[1])
    near("db", db, want[2], 70 * EPS * mag[2])
    near("dinitial", dh, want[3], 6 * EPS * mag[3] + out * np.abs(want[3]))


def test_conv_more_blocks_than_a_grid_has():
    """Launches of more than 2^32 threads: many sequences of one token, and many channels."""
    N, D, W = 2 ** 26 + 4, 33, 2
    x, w = torch.full((N, 1, D), 0.5, dtype=BF, device=DEV), randn(gen(13), D, W, dtype=BF)
    x[-4:] = 2.0
    y, _ = kda.kda_conv_fwd(x, w, activation=None)
    want = (w[:, 1].float()[None] * x[:, 0, :1].float()[[0, -1]]).to(BF)
    assert torch.equal(y[-4:, 0], want[1].expand(4, -1)) and torch.equal(y[0, 0], want[0])
    assert torch.equal(y[N // 2], y[0]) and torch.equal(y[2 ** 26 - 1], y[0])
    del x, y
    D = 2 ** 27 // 3 + 61
    x, dy, w = (randn(gen(14 + i), *s, dtype=BF) for i, s in enumerate([(1, 1, D), (1, 1, D), (D, W)]))
    dx, dw, db, _ = kda.kda_conv_bwd(dy, x, w, w[:, 0].contiguous(), activation=None)
    assert torch.equal(dw[:, 1], (dy.float() * x.float())[0, 0]) and not dw[:, 0].any() and torch.equal(db, dy.float()[0, 0])
    assert torch.equal(dx, (dy.float() * w[:, 1].float()).to(BF))


# ------------------------------------------------------------------------------ the norm
def test_norm_more_rows_than_a_grid_has():
    rows = 2 ** 28 + 16     # sixteen a block of 256 threads
    x = torch.full((rows, 1), 2.0, dtype=BF, device=DEV)
    x[-16:] = -3.0
    y, _, r = kda.kda_rmsnorm_fwd(x, torch.ones(1, dtype=BF, device=DEV), eps=0.0, output_rstd=True)
    assert (y[:-16] == 1).all() and (y[-16:] == -1).all() and (r[:-16] == 0.5).all() and (r[-16:] == np.float32(1 / 3)).all()
    q, s, _ = kda.kda_rmsnorm_quant_fwd(x, torch.ones(1, dtype=BF, device=DEV), eps=0.0)
    assert (q[-16:].float() == -448).all() and (q[::4099].float().abs() == 448).all() and (s[::4099] == np.float32(1 / 448)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_codes_are_those_of_the_quotient(group, dtype):
    """Rows of +-1 and eps 0 have r = 1 exactly, so y is the weight: the codes are e4m3 of the fp32
    quotient y / s, here for weights at and beside every tie between codes."""
    D, rows = 1024, 3
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    ties = (codes[:-1] + codes[1:]) / 2
    rng = np.random.default_rng(50)
    w = torch.empty(D)
    for at in range(0, D, 128):
        top = np.float32(rng.uniform(0.5, 2.0))
        s = np.float32(top / np.float32(448))
        v = (ties[torch.tensor(rng.permutation(126)[:127])].numpy() * s).astype(np.float32)
        v = v.view(np.int32) + rng.integers(-2, 3, v.size).astype(np.int32)
        w[at:at + 128] = torch.tensor(np.concatenate([[top, -top], v.view(np.float32)]).astype(np.float32))
    if not group:
        w[128:] = w[:128].repeat(D // 128 - 1)
    sign = torch.where(torch.rand(rows, D, generator=torch.Generator().manual_seed(1)) < 0.5, -1.0, 1.0)
    q, s, _ = kda.kda_rmsnorm_quant_fwd(sign.to(DEV, dtype), w.to(DEV), eps=0.0, group=group)
    y = sign * w
    ws = y.view(rows, -1, group or D).abs().amax(-1) / 448.0
    assert torch.equal(s.cpu().view(ws.shape), ws)
    want = (y.view(rows, -1, group or D) / ws[..., None]).to(torch.float8_e4m3fn).view(rows, D)
    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))


# ------------------------------------------------------------------------- outputs given
def test_overlapping_outputs_are_refused():
    def refused(f, *a, **k):
        with pytest.raises(ValueError, match="overlap"):
            f(*a, **k)
    c = conv_case(60, BF, BF, 4, 64, B=2, T=40)
    flat = torch.zeros(3 * 5120, dtype=BF, device=DEV)
    c["x"] = flat[:5120].view(2, 40, 64)
    out = flat[5120:10240].view(2, 40, 64)
    refused(kda.kda_conv_fwd, **c, out=flat[5056:10176].view(2, 40, 64))             # x's last row
    refused(kda.kda_conv_fwd, **c, output_final_state=True, final_state=flat[:384].view(2, 3, 64))
    refused(kda.kda_conv_fwd, **c, out=out, output_final_state=True, final_state=flat[9856:10240].view(2, 3, 64))
    refused(kda.kda_conv_bwd, out, **c, workspace=flat[5120:10240])
    kda.kda_conv_fwd(**c, out=out, output_final_state=True, final_state=c["initial_state"])
    kda.kda_conv_fwd(**c, out=out, output_final_state=True, final_state=flat[10240:10624].view(2, 3, 64))
    states = torch.zeros(2 * 16384, device=DEV)
    s = ssm_case(61, BF, 1, 2, 64, 64, T=40, B=2)
    s["initial_state"] = states[:16384].view(2, 2, 64, 64)
    for f in SCANS:
        refused(f, **s, output_final_state=True, final_state=states[64:64 + 16384].view(2, 2, 64, 64))
        refused(f, **s, out=s["x"])
        f(**s, output_final_state=True, final_state=s["initial_state"])
        f(**s, output_final_state=True, final_state=states[16384:].view(2, 2, 64, 64))
    refused(kda.kda_ssm_chunk_fwd, **s, workspace=states)
    both = torch.zeros(2 * 16384, device=DEV)
    s = ssm_case(62, F32, 1, 2, 64, 64, T=128)
    for f in SCANS:
        refused(f, **s, out=both[:16384].view(1, 128, 2, 64), output_final_state=True, final_state=both[8192:16384].view(1, 2, 64, 64))
    # between the rows of a wider tensor there is room for others
    wide = torch.zeros(3, 4096, dtype=BF, device=DEV)
    x, w = wide[:, :64], randn(gen(66), 64, dtype=BF)
    kda.kda_rmsnorm_fwd(x, w, out=wide[1, 64:256].view(3, 64))
    refused(kda.kda_rmsnorm_fwd, x, w, out=wide[1, 63:255].view(3, 64))
    refused(kda.kda_rmsnorm_fwd, x, w, out=wide.view(-1)[2 * 4096 - 191:2 * 4096 + 1].view(3, 64))
    kda.kda_rmsnorm_fwd(x, w, out=wide.view(-1)[2 * 4096 - 192:2 * 4096].view(3, 64))
    # the norms
    n, w = randn(gen(63), 9, 512, dtype=BF), randn(gen(64), 256, dtype=BF)
    x, res = n[:, :256], randn(gen(65), 9, 256, dtype=BF)
    over = n.view(-1)[:9 * 256].view(9, 256)
    t = torch.empty(9, 256, dtype=BF, device=DEV)
    for f in (kda.kda_rmsnorm_fwd, kda.kda_rmsnorm_quant_fwd):
        refused(f, x, w, res, residual_out=over)
    refused(kda.kda_rmsnorm_fwd, x, w, res, out=over)
    refused(kda.kda_rmsnorm_fwd, x, w, res, out=t, residual_out=t)
    refused(kda.kda_rmsnorm_fwd, x, w, res, out=res, residual_out=res)
    refused(kda.kda_rmsnorm_fwd, x[:1], w, out=w.view(1, 256))
    q = torch.empty(9, 256, dtype=torch.float8_e4m3fn, device=DEV)
    refused(kda.kda_rmsnorm_quant_fwd, x, w, out=q, scales=q.view(torch.uint8).view(-1)[:36].view(torch.float32).view(9, 1))
    refused(kda.kda_rmsnorm_quant_fwd, x, w, res, out=res.view(torch.uint8).view(-1)[:2304].view(9, 256).view(torch.float8_e4m3fn))
    refused(kda.kda_rmsnorm_bwd, t, res, w, torch.ones(9, device=DEV), workspace=res)
    # in place, row for row: each of y and h over either input
    a = x.contiguous()
    y, h, _ = kda.kda_rmsnorm_fwd(a, w, res)
    for swap in (False, True):
        b, r = a.clone(), res.clone()
        y2, h2, _ = kda.kda_rmsnorm_fwd(b, w, r, out=r if swap else b, residual_out=b if swap else r)
        assert torch.equal(y, y2) and torch.equal(h, h2)
