"""Refusals and sizes of the operators around the mixer, without a GPU: bad arguments are
turned down on the host before anything is enqueued, by the C entry points and by the
binding."""
import os

import pytest
import torch

import gated_delta_rule_64_amd as kda
from gated_delta_rule_64_amd import _layer, _lib

P = 1 << 20     # a pointer-like value that no refused call follows
OK, NULL, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE, ARG = 0, -1, -2, -3, -4, -5, -7


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.library_path()):
        from gated_delta_rule_64_amd import build
        build.build()
    return _layer._load()


def conv_fwd(lib, **kw):
    a = dict(x=P, x_stride=64, w=P, bias=None, h0=None, cu=None, N=2, y=P, hT=None, B=2, T=5, D=64, W=4, dt=1, wdt=1, act=1)
    a.update(kw)
    return lib.kda_conv_fwd(*a.values(), None, None)


def conv_bwd(lib, **kw):
    a = dict(dy=P, x=P, x_stride=64, w=P, bias=None, h0=None, cu=None, N=2, df=None, dx=P, dw=P, db=None, dh0=None, B=2,
             T=5, D=64, W=4, dt=1, wdt=1, act=1, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.kda_conv_bwd(*a.values(), None, None)


@pytest.mark.parametrize("call", [conv_fwd, conv_bwd])
@pytest.mark.parametrize("kw,code,word", [
    (dict(dt=2), DTYPE, "dtype"), (dict(wdt=-1), DTYPE, "dtype"), (dict(act=2), ARG, "activation"),
    (dict(B=-1), SHAPE, "non-negative"), (dict(N=3), SHAPE, "N must equal B"), (dict(cu=P), SHAPE, "B == 1"),
    (dict(D=0), SHAPE, "D"), (dict(W=1), UNSUPPORTED, "W"), (dict(W=5), UNSUPPORTED, "W"),
    (dict(x_stride=63), SHAPE, "x_stride"), (dict(x_stride=1 << 40), SHAPE, "x_stride"), (dict(x=None), NULL, "x"),
    (dict(w=None), NULL, "weight"), (dict(B=1 << 16, N=1 << 16, T=1 << 16), SHAPE, "2^31"),
])
def test_conv_refusals(lib, call, kw, code, word):
    assert call(lib, **kw) == code
    assert word in kda.kda_last_error()


def test_conv_more_refusals(lib):
    assert conv_fwd(lib, y=None) == NULL
    assert conv_bwd(lib, dy=None) == NULL
    assert conv_bwd(lib, dx=None) == NULL
    assert conv_bwd(lib, dw=None) == NULL
    need = lib.kda_conv_bwd_workspace_bytes(2, 5, 64, 4, 2, 0, 1)
    assert need > 0
    assert conv_bwd(lib, wsb=need - 1) == WORKSPACE
    assert conv_bwd(lib, ws=None) == WORKSPACE
    assert conv_bwd(lib, ws=P + 4) == WORKSPACE
    for bad in ((-1, 5, 64, 4, 2, 0, 1), (2, 5, 0, 4, 2, 0, 1), (2, 5, 64, 5, 2, 0, 1), (2, 5, 64, 4, 2, 0, 7)):
        assert lib.kda_conv_bwd_workspace_bytes(*bad) == 0
    # no sequences: nothing to do
    assert conv_fwd(lib, B=0, N=0) == OK


def ssm(lib, chunk, **kw):
    a = dict(x=P, xs=512, dt=P, dts=4, A=P, b=P, bs=256, c=P, cs=256, D=None, bias=None, h0=None, cu=None, N=2, y=P,
             hT=None, B=2, T=5, H=2, HV=4, K=128, V=128, dtype=1, dtdt=1, sp=1)
    ws = [kw.pop("ws", P), kw.pop("wsb", 1 << 40)]
    a.update(kw)
    if chunk:
        return lib.kda_ssm_chunk_fwd(*a.values(), *ws, None, None)
    return lib.kda_ssm_recurrent_fwd(*a.values(), None, None)


@pytest.mark.parametrize("chunk", [True, False])
@pytest.mark.parametrize("kw,code,word", [
    (dict(dtype=3), DTYPE, "dtype"), (dict(dtdt=9), DTYPE, "dtype"), (dict(T=-1), SHAPE, "non-negative"),
    (dict(N=1), SHAPE, "N must equal B"), (dict(cu=P), SHAPE, "B == 1"), (dict(H=0), SHAPE, "positive"),
    (dict(H=3), SHAPE, "multiple of H"), (dict(K=32), UNSUPPORTED, "K"), (dict(V=96), UNSUPPORTED, "V"),
    (dict(xs=511), SHAPE, "x_stride"), (dict(xs=516), SHAPE, "16 bytes"), (dict(dts=3), SHAPE, "dt_stride"),
    (dict(bs=255), SHAPE, "b_stride"), (dict(cs=260), SHAPE, "16 bytes"), (dict(x=None), NULL, "x"),
    (dict(A=None), NULL, "A_log"), (dict(y=None), NULL, "y"), (dict(h0=P + 4), SHAPE, "aligned"),
    (dict(b=P + 2), SHAPE, "aligned"), (dict(B=1 << 20, N=1 << 20, T=1 << 20), SHAPE, "2^31"),
    (dict(B=1 << 28, N=1 << 28, T=1, HV=16, H=2, xs=2048, dts=16), SHAPE, "too large"),
])
def test_ssm_refusals(lib, chunk, kw, code, word):
    assert ssm(lib, chunk, **kw) == code
    assert word in kda.kda_last_error()


def test_ssm_workspace_sizes(lib):
    f = lib.kda_ssm_chunk_fwd_workspace_bytes
    for bad in ((-1, 5, 2, 4, 128, 128, 2, 0, 1), (2, 5, 3, 4, 128, 128, 2, 0, 1), (2, 5, 2, 4, 96, 128, 2, 0, 1),
                (2, 5, 2, 4, 128, 100, 2, 0, 1), (2, 5, 2, 4, 128, 128, 2, 0, 5)):
        assert f(*bad) == 0
    need = f(1, 8192, 1, 4, 128, 128, 1, 0, 1)
    if need:
        args = dict(B=1, N=1, T=8192, H=1, bs=128, cs=128)
        assert ssm(lib, True, ws=None, **args) == WORKSPACE
        assert ssm(lib, True, wsb=need - 1, **args) == WORKSPACE
        assert ssm(lib, True, ws=P + 16, **args) == WORKSPACE
    assert ssm(lib, True, B=0, N=0) == OK and ssm(lib, False, B=0, N=0) == OK


def norm(lib, **kw):
    a = dict(x=P, xs=256, w=P, res=None, y=P, h=None, rstd=None, rows=3, D=256, eps=1e-6, dt=1, wdt=1)
    a.update(kw)
    return lib.kda_rmsnorm_fwd(*a.values(), None)


def quant(lib, **kw):
    a = dict(x=P, xs=256, w=P, res=None, q=P, s=P, h=None, rows=3, D=256, group=128, eps=1e-6, dt=1, wdt=1)
    a.update(kw)
    return lib.kda_rmsnorm_quant_fwd(*a.values(), None)


@pytest.mark.parametrize("call", [norm, quant])
@pytest.mark.parametrize("kw,code,word", [
    (dict(dt=4), DTYPE, "dtype"), (dict(rows=-1), SHAPE, "rows"), (dict(rows=1 << 40), SHAPE, "rows"),
    (dict(D=0), SHAPE, "D"), (dict(xs=255), SHAPE, "x_stride"), (dict(eps=-1.0), ARG, "eps"),
    (dict(eps=float("nan")), ARG, "eps"), (dict(D=65664, xs=65664), UNSUPPORTED, "65536"),
    (dict(D=9001, xs=9001), UNSUPPORTED, "8192"), (dict(x=None), NULL, "x"), (dict(w=None), NULL, "weight"),
])
def test_norm_refusals(lib, call, kw, code, word):
    assert call(lib, **kw) == code
    assert word in kda.kda_last_error()


def test_quant_refusals(lib):
    assert quant(lib, group=64) == UNSUPPORTED
    assert quant(lib, group=0) == UNSUPPORTED
    assert quant(lib, D=200, xs=200) == UNSUPPORTED
    assert quant(lib, x=P + 2) == UNSUPPORTED and "aligned" in kda.kda_last_error()
    assert quant(lib, xs=260) == UNSUPPORTED
    assert quant(lib, s=None) == NULL
    assert quant(lib, rows=0) == OK and norm(lib, rows=0) == OK


def test_norm_bwd_refusals(lib):
    def bwd(**kw):
        a = dict(dy=P, h=P, w=P, rstd=P, dh=None, dx=P, dw=P, rows=3, D=256, dt=1, wdt=1, ws=P, wsb=1 << 30)
        a.update(kw)
        return lib.kda_rmsnorm_bwd(*a.values(), None)
    assert bwd(dt=8) == DTYPE
    assert bwd(rows=-2) == SHAPE
    assert bwd(D=70000) == UNSUPPORTED
    for name in ("dy", "h", "w", "rstd", "dx", "dw"):
        assert bwd(**{name: None}) == NULL
    need = lib.kda_rmsnorm_bwd_workspace_bytes(3, 256, 1)
    assert need >= 256 * 4
    assert bwd(wsb=need - 1) == WORKSPACE and bwd(ws=None) == WORKSPACE and bwd(ws=P + 8) == WORKSPACE
    assert lib.kda_rmsnorm_bwd_workspace_bytes(-1, 256, 1) == 0
    assert lib.kda_rmsnorm_bwd_workspace_bytes(3, 1 << 20, 1) == 0


# ---------------------------------------------------------------- the binding's own checks
def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_constants_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kda.h")).read()
    assert "KDA_ACT_NONE = %d" % kda.KDA_ACT_NONE in text and "KDA_ACT_SILU = %d" % kda.KDA_ACT_SILU in text


@pytest.mark.parametrize("args,kw,err", [
    ((bf(2, 5), bf(64, 4)), {}, ValueError),
    ((bf(2, 5, 64), bf(63, 4)), {}, ValueError),
    ((bf(2, 5, 64), bf(64, 4)), dict(activation="relu"), ValueError),
    ((bf(2, 5, 64).half(), bf(64, 4)), {}, TypeError),
    ((bf(2, 5, 64), bf(64, 4).double()), {}, TypeError),
    ((bf(2, 5, 64), bf(64, 4)), dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), ValueError),
    ((bf(1, 5, 64), bf(64, 4)), dict(cu_seqlens=torch.zeros(3, dtype=torch.int64)), TypeError),
    ((bf(1, 5, 64), bf(64, 4)), dict(cu_seqlens=torch.zeros(0, dtype=torch.int32)), ValueError),
    ((bf(2, 64, 5).transpose(1, 2), bf(64, 4)), {}, ValueError),
    ((bf(2, 9, 64)[:, ::2], bf(64, 4)), {}, ValueError),           # rows of the two batches unevenly spaced
    ((bf(1, 1, 64).expand(2, 5, 64), bf(64, 4)), {}, ValueError),  # rows on top of each other
    ((bf(2, 5, 64), bf(64, 4)), {}, ValueError),                   # not on a GPU
])
def test_conv_binding_refusals(lib, args, kw, err):
    with pytest.raises(err):
        kda.kda_conv_fwd(*args, **kw)
    with pytest.raises(err):
        kda.kda_conv_bwd(args[0], *args, **kw)


def test_ssm_binding_refusals(lib):
    def call(**kw):
        a = dict(x=bf(2, 5, 4, 64), dt=bf(2, 5, 4), A_log=torch.zeros(4), b=bf(2, 5, 2, 64), c=bf(2, 5, 2, 64))
        a.update(kw)
        for f in (kda.kda_ssm_chunk_fwd, kda.kda_ssm_recurrent_fwd):
            with pytest.raises((ValueError, TypeError)) as e:
                f(**a)
        return str(e.value)
    assert "GPU" in call()
    assert "x takes" in call(x=bf(2, 5, 64))
    assert "dt" in call(dt=bf(2, 5, 3))
    assert "c" in call(c=bf(2, 5, 4, 64))
    assert "dtype" in call(b=torch.zeros(2, 5, 2, 64))
    assert "dtype" in call(dt=torch.zeros(2, 5, 4, dtype=torch.float16))
    assert "contiguous" in call(x=bf(2, 5, 64, 4).transpose(2, 3))


def test_norm_binding_refusals(lib):
    w = bf(256)
    for call in (lambda **k: kda.kda_rmsnorm_fwd(bf(3, 256), w, **k), lambda **k: kda.kda_rmsnorm_quant_fwd(bf(3, 256), w, **k)):
        with pytest.raises(ValueError):
            call()                                   # not on a GPU
        with pytest.raises(ValueError):
            call(residual=bf(2, 256))
    with pytest.raises(ValueError):
        kda.kda_rmsnorm_fwd(bf(3, 255), w)
    with pytest.raises(ValueError):
        kda.kda_rmsnorm_quant_fwd(bf(3, 256), w, group=64)
    with pytest.raises(TypeError):
        kda.kda_rmsnorm_bwd(torch.zeros(3, 256), bf(3, 256).half(), w, torch.zeros(3))


def test_row_strides():
    f = _layer._row_stride
    wide = torch.zeros(2, 6, 40)
    assert f("x", wide[:, :, 8:24], 2) == 40
    assert f("x", wide[:, 2:3, 8:24], 2) == 240          # one token of each sequence
    assert f("x", wide[:1, 2:3, 8:24], 2) == 16
    assert f("x", wide[:1], 2) == 40
    assert f("x", torch.zeros(2, 0, 40), 2) == 40
    assert f("x", wide.view(2, 6, 4, 10), 2) == 40
    line = torch.zeros(8)
    assert f("x", line, 0) == 8
    with pytest.raises(ValueError):
        f("x", line[::2], 0)                             # one row whose elements are apart
    with pytest.raises(ValueError):
        f("x", torch.zeros(4)[::2], 0)
    with pytest.raises(ValueError):
        f("x", wide[:, 1:], 2)
    with pytest.raises(ValueError):
        f("x", wide[..., ::2], 2)
