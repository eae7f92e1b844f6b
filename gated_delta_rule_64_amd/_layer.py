"""Binding of the operators around the mixer: the short causal convolution, the selective
state space scan and the RMS norm (see ``include/kda.h`` for the contract)."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import KDA_BF16, KDA_F32, KdaError, _debug_raise, _debug_status

KDA_ACT_NONE = 0
KDA_ACT_SILU = 1

_CODES = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}
_ACTIVATIONS = {None: KDA_ACT_NONE, "silu": KDA_ACT_SILU}
_funcs = None


def _load():
    """The library with this module's entry points typed."""
    global _funcs
    if _funcs is not None:
        return _funcs
    lib = _lib.load_library()
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
    seqs = [vp, vp, i32]                       # initial_state, cu_seqlens, N
    ssm = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, *seqs, vp, vp] + [i32] * 9
    for name, args in (
            ("kda_conv_fwd", [vp, i64, vp, vp, *seqs, vp, vp] + [i32] * 7 + [vp, vp]),
            ("kda_conv_bwd", [vp, vp, i64, vp, vp, *seqs, vp, vp, vp, vp, vp] + [i32] * 7 + [vp, sz, vp, vp]),
            ("kda_ssm_chunk_fwd", ssm + [vp, sz, vp, vp]),
            ("kda_ssm_recurrent_fwd", ssm + [vp, vp]),
            ("kda_rmsnorm_fwd", [vp, i64, vp, vp, vp, vp, vp, i64, i32, f32, i32, i32, vp]),
            ("kda_rmsnorm_quant_fwd", [vp, i64, vp, vp, vp, vp, vp, i64, i32, i32, f32, i32, i32, vp]),
            ("kda_rmsnorm_bwd", [vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, vp, sz, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = i32, args
    for name, args in (("kda_conv_bwd_workspace_bytes", [i32] * 7),
                       ("kda_ssm_chunk_fwd_workspace_bytes", [i32] * 9),
                       ("kda_rmsnorm_bwd_workspace_bytes", [i64, i32, i32])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = sz, args
    _funcs = lib
    return lib


def _code(t, what):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} has dtype {t.dtype}; the library takes bfloat16 or float32")
    return code


def _at(t):
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object around it (2 us of an 11 us call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(dev, fn, *args):
    """``fn(*args, stream)`` on ``dev``'s current stream, with ``dev`` current."""
    if dev.index == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev.index))
    if rc != 0:
        raise KdaError(rc, _lib.kda_last_error())


def _want(name, t, shape, dtypes, dev=None):
    """``t``, unless None, has this shape and one of these dtypes; with ``dev``, it is
    contiguous and there."""
    if t is None:
        return
    if t.shape != shape:
        raise ValueError(f"{name}: got shape {tuple(t.shape)}, this problem needs {tuple(shape)}")
    if t.dtype not in dtypes:
        names = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise TypeError(f"{name}: got dtype {str(t.dtype).replace('torch.', '')}, expected {names}")
    if dev is not None:
        if t.device != dev:
            _placed(name, t, dev)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _placed(name, t, dev):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")


_FLOAT = (torch.bfloat16, torch.float32)
_F32 = (torch.float32,)


def _row_stride(name, t, lead):
    """Elements between consecutive rows of ``t``, whose first ``lead`` axes count rows and
    whose others are a row, contiguous inside; the rows evenly spaced."""
    shape = t.shape
    width = 1
    for n in shape[lead:]:
        width *= n
    if t.is_contiguous():
        return width
    strides = t.stride()
    inner = 1
    for d in range(len(shape) - 1, lead - 1, -1):
        if shape[d] != 1 and strides[d] != inner:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        inner *= shape[d]
    stride, span = None, None
    for d in range(lead - 1, -1, -1):
        if shape[d] == 1:
            continue
        if stride is None:
            stride = strides[d]
        elif strides[d] != span:
            raise ValueError(f"{name}: rows must be evenly spaced over the leading axes")
        span = strides[d] * shape[d]
    if stride is None:
        return width
    if stride < width:
        raise ValueError(f"{name}: rows must not overlap")
    return stride


def _sequences(B, cu_seqlens):
    if cu_seqlens is None:
        return B
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens: got dtype %s, expected int32" % str(cu_seqlens.dtype).replace("torch.", ""))
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens: expected a 1-D tensor of N + 1 offsets")
    if B != 1:
        raise ValueError("cu_seqlens packs sequences into one row: B must be 1")
    return cu_seqlens.numel() - 1


def _status(dev, dev_status, cu_seqlens, debug):
    if cu_seqlens is not None:
        _placed("cu_seqlens", cu_seqlens, dev)
        if not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous")
    if dev_status is not None:
        if dev_status.dtype != torch.int32 or dev_status.numel() < 1:
            raise TypeError("dev_status: expected an int32 tensor with at least one element")
        _placed("dev_status", dev_status, dev)
    return _debug_status(debug, dev_status, dev)


def _bytes(name, workspace, need, dev):
    """The caller's workspace, or a new one of ``need`` bytes."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _placed(name, workspace, dev)
    if not workspace.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return workspace


def _apart(name, out, others, same=()):
    """A buffer a caller gives to be written shares no byte with the tensors in ``others``
    (name, tensor or None, rows, elements between rows), except one named in ``same`` at its
    very place, whose elements are read before they are written. Between rows that are apart there
    may be other tensors."""
    begin, size = out.data_ptr(), out.numel() * out.element_size()
    for other, t, rows, stride in others:
        if t is None or size == 0 or t.numel() == 0:
            continue
        at, item = t.data_ptr(), t.element_size()
        if begin == at and other in same and t.is_contiguous():
            continue
        width, step = t.numel() // rows * item, stride * item
        # the rows that end behind the buffer's begin and start ahead of its end
        if max(0, (begin - at - width) // step + 1) <= min(rows - 1, (begin + size - 1 - at) // step):
            raise ValueError(f"{name} must not overlap {other}")


def _whole(**tensors):
    """Contiguous tensors, as ``_apart`` takes them."""
    return tuple((name, t, 1, 1) for name, t in tensors.items())


def _size(t):
    return 0 if t is None else t.numel() * t.element_size()


# ------------------------------------------------------------------- the short convolution
def _conv_inputs(x, weight, bias, initial_state, cu_seqlens, activation):
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    if x.dim() != 3:
        raise ValueError("x takes [B, T, D]")
    B, T, D = x.shape
    code, w_code = _code(x, "x"), _code(weight, "weight")
    if weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError(f"weight: got shape {tuple(weight.shape)}, this problem needs ({D}, W)")
    W = weight.shape[1]
    N = _sequences(B, cu_seqlens)
    dev = x.device
    stride = _row_stride("x", x, 2)
    _placed("x", x, dev)
    _want("weight", weight, (D, W), _FLOAT, dev)
    _want("bias", bias, (D,), (weight.dtype,), dev)
    _want("initial_state", initial_state, (N, W - 1, D), (x.dtype,), dev)
    return B, T, D, W, N, code, w_code, stride, dev


def kda_conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, output_final_state=False,
                 *, activation="silu", out=None, final_state=None, dev_status=None, debug=False):
    """Short causal depthwise convolution with bias and activation ("silu" or None), ahead
    of the mixer. Returns ``(y, final_state or None)``.

    ``x`` [B, T, D] (bfloat16 or float32; columns of a wider tensor are taken as they are),
    ``weight`` [D, W] with W of 2 to 4, the last tap the token's own; ``bias`` [D] in
    weight's dtype. ``initial_state`` [N, W-1, D] in x's dtype: the rows before each
    sequence's first token, oldest first (zeros without one); the final state is the same
    of its last rows and may be written into ``initial_state`` itself. A decode step is
    T = 1. ``out``, ``dev_status`` and ``debug`` as in ``kda_chunk_fwd``."""
    lib = _load()
    B, T, D, W, N, code, w_code, stride, dev = _conv_inputs(x, weight, bias, initial_state, cu_seqlens, activation)
    if out is not None or final_state is not None:
        inputs = (("x", x, B * T, stride), *_whole(weight=weight, bias=bias, initial_state=initial_state,
                                                   cu_seqlens=cu_seqlens))
    if out is None:
        out = x.new_empty((B, T, D))
    else:
        _want("out", out, (B, T, D), (x.dtype,), dev)
        _apart("out", out, inputs)
    if not output_final_state:
        final_state = None
    elif final_state is None:
        final_state = x.new_empty((N, W - 1, D))
    else:
        _want("final_state", final_state, (N, W - 1, D), (x.dtype,), dev)
        _apart("final_state", final_state, inputs + _whole(out=out), same=("initial_state",))
    dev_status = _status(dev, dev_status, cu_seqlens, debug)
    _call(dev, lib.kda_conv_fwd, _at(x), stride, _at(weight), _at(bias), _at(initial_state), _at(cu_seqlens), N,
          _at(out), _at(final_state), B, T, D, W, code, w_code, _ACTIVATIONS[activation], _at(dev_status))
    _debug_raise(debug, dev_status, dev)
    return out, final_state


def kda_conv_bwd_workspace_bytes(B, T, D, W, N, packed, dtype=KDA_BF16) -> int:
    if isinstance(dtype, torch.dtype):
        dtype = _CODES[dtype]
    return int(_load().kda_conv_bwd_workspace_bytes(B, T, D, W, N, int(bool(packed)), int(dtype)))


def kda_conv_bwd(dy, x, weight, bias=None, initial_state=None, cu_seqlens=None, dfinal_state=None,
                 *, activation="silu", workspace=None, dev_status=None, debug=False):
    """Gradients of ``kda_conv_fwd``. ``dy`` [B, T, D] in x's dtype, ``dfinal_state``
    [N, W-1, D] or None. Returns ``(dx, dweight, dbias, dinitial_state)``: dweight [D, W]
    and dbias [D] float32 (dbias None without a bias, dinitial_state None without an
    initial state). Rows of dx outside every sequence are zero."""
    lib = _load()
    B, T, D, W, N, code, w_code, stride, dev = _conv_inputs(x, weight, bias, initial_state, cu_seqlens, activation)
    _want("dy", dy, (B, T, D), (x.dtype,), dev)
    _want("dfinal_state", dfinal_state, (N, W - 1, D), (x.dtype,), dev)
    new = torch.empty if cu_seqlens is None else torch.zeros
    dx = new(B, T, D, dtype=x.dtype, device=dev)
    dweight = torch.empty(D, W, dtype=torch.float32, device=dev)
    dbias = torch.empty(D, dtype=torch.float32, device=dev) if bias is not None else None
    dinitial = new(N, W - 1, D, dtype=x.dtype, device=dev) if initial_state is not None else None
    if workspace is not None:
        _apart("workspace", workspace, (("x", x, B * T, stride),
                                        *_whole(dy=dy, weight=weight, bias=bias, initial_state=initial_state,
                                                cu_seqlens=cu_seqlens, dfinal_state=dfinal_state)))
    workspace = _bytes("workspace", workspace,
                       lib.kda_conv_bwd_workspace_bytes(B, T, D, W, N, int(cu_seqlens is not None), code), dev)
    dev_status = _status(dev, dev_status, cu_seqlens, debug)
    _call(dev, lib.kda_conv_bwd, _at(dy), _at(x), stride, _at(weight), _at(bias), _at(initial_state),
          _at(cu_seqlens), N, _at(dfinal_state), _at(dx), _at(dweight), _at(dbias), _at(dinitial), B, T, D, W, code,
          w_code, _ACTIVATIONS[activation], _at(workspace), _size(workspace), _at(dev_status))
    _debug_raise(debug, dev_status, dev)
    return dx, dweight, dbias, dinitial


# ---------------------------------------------------------------- the state space scan
def _ssm(chunk, x, dt, A_log, b, c, D, dt_bias, initial_state, cu_seqlens, output_final_state, dt_softplus, out,
         final_state, workspace, dev_status, debug):
    lib = _load()
    if x.dim() != 4 or b.dim() != 4:
        raise ValueError("x takes [B, T, HV, V] and b and c [B, T, H, K]")
    B, T, HV, V = x.shape
    H, K = b.shape[2:]
    code, dt_code = _code(x, "x"), _code(dt, "dt")
    N = _sequences(B, cu_seqlens)
    dev = x.device
    _want("dt", dt, (B, T, HV), _FLOAT)
    _want("b", b, (B, T, H, K), (x.dtype,))
    _want("c", c, (B, T, H, K), (x.dtype,))
    strides = [_row_stride(name, t, 2) for name, t in (("x", x), ("dt", dt), ("b", b), ("c", c))]
    for name, t in (("x", x), ("dt", dt), ("b", b), ("c", c)):
        _placed(name, t, dev)
    _want("A_log", A_log, (HV,), _F32, dev)
    _want("D", D, (HV,), _F32, dev)
    _want("dt_bias", dt_bias, (HV,), _F32, dev)
    _want("initial_state", initial_state, (N, HV, K, V), _F32, dev)
    if out is not None or final_state is not None or workspace is not None:
        inputs = (*((name, t, B * T, s) for (name, t), s in zip((("x", x), ("dt", dt), ("b", b), ("c", c)), strides)),
                  *_whole(A_log=A_log, D=D, dt_bias=dt_bias, initial_state=initial_state, cu_seqlens=cu_seqlens))
    if out is None:
        out = x.new_empty((B, T, HV, V))
    else:
        _want("out", out, (B, T, HV, V), (x.dtype,), dev)
        _apart("out", out, inputs)
    if not output_final_state:
        final_state = None
    elif final_state is None:
        final_state = A_log.new_empty((N, HV, K, V))
    else:
        _want("final_state", final_state, (N, HV, K, V), _F32, dev)
        _apart("final_state", final_state, inputs + _whole(out=out), same=("initial_state",))
    dev_status = _status(dev, dev_status, cu_seqlens, debug)
    args = [_at(x), strides[0], _at(dt), strides[1], _at(A_log), _at(b), strides[2], _at(c), strides[3], _at(D),
            _at(dt_bias), _at(initial_state), _at(cu_seqlens), N, _at(out), _at(final_state), B, T, H, HV, K, V, code,
            dt_code, int(bool(dt_softplus))]
    if chunk:
        need = lib.kda_ssm_chunk_fwd_workspace_bytes(B, T, H, HV, K, V, N, int(cu_seqlens is not None), code)
        if workspace is not None:
            _apart("workspace", workspace, inputs + _whole(out=out, final_state=final_state))
        workspace = _bytes("workspace", workspace, need, dev)
        _call(dev, lib.kda_ssm_chunk_fwd, *args, _at(workspace), _size(workspace), _at(dev_status))
    else:
        _call(dev, lib.kda_ssm_recurrent_fwd, *args, _at(dev_status))
    _debug_raise(debug, dev_status, dev)
    return out, final_state


def kda_ssm_chunk_fwd(x, dt, A_log, b, c, D=None, dt_bias=None, initial_state=None, cu_seqlens=None,
                      output_final_state=False, *, dt_softplus=False, out=None, final_state=None, workspace=None,
                      dev_status=None, debug=False):
    """Selective state space scan over prompts, in chunks of 64 tokens. Returns
    ``(y, final_state or None)``.

    S <- exp(-exp(A_log) dt') S + b (dt' x)^T and y = S^T c + D x per head, with
    dt' = softplus(dt + dt_bias) under ``dt_softplus``, else dt + dt_bias. ``x``
    [B, T, HV, V]; ``dt`` [B, T, HV] (bfloat16 or float32); ``b``, ``c`` [B, T, H, K] shared
    by HV / H heads each, in x's dtype (all four may be columns of a wider tensor);
    ``A_log``, ``D``, ``dt_bias`` float32 [HV]; states float32 [N, HV, K, V]. K is 64 or
    128, V a multiple of 64. The other arguments as in ``kda_chunk_fwd``."""
    return _ssm(True, x, dt, A_log, b, c, D, dt_bias, initial_state, cu_seqlens, output_final_state, dt_softplus, out,
                final_state, workspace, dev_status, debug)


def kda_ssm_chunk_fwd_workspace_bytes(B, T, H, HV, K, V, N, packed, dtype=KDA_BF16) -> int:
    if isinstance(dtype, torch.dtype):
        dtype = _CODES[dtype]
    return int(_load().kda_ssm_chunk_fwd_workspace_bytes(B, T, H, HV, K, V, N, int(bool(packed)), int(dtype)))


def kda_ssm_recurrent_fwd(x, dt, A_log, b, c, D=None, dt_bias=None, initial_state=None, cu_seqlens=None,
                          output_final_state=False, *, dt_softplus=False, out=None, final_state=None,
                          dev_status=None, debug=False):
    """The scan of ``kda_ssm_chunk_fwd`` token by token (decode, short prompts): the same
    arguments and results, without a workspace."""
    return _ssm(False, x, dt, A_log, b, c, D, dt_bias, initial_state, cu_seqlens, output_final_state, dt_softplus, out,
                final_state, None, dev_status, debug)


# ---------------------------------------------------------------------------- the norm
def _norm_inputs(x, weight, residual):
    if x.dim() < 1:
        raise ValueError("x takes [..., D]")
    D = x.shape[-1]
    code, w_code = _code(x, "x"), _code(weight, "weight")
    dev = x.device
    stride = _row_stride("x", x, x.dim() - 1)
    _placed("x", x, dev)
    _want("weight", weight, (D,), _FLOAT, dev)
    shape = tuple(x.shape)
    _want("residual", residual, shape, (x.dtype,), dev)
    rows = x.numel() // D if D else 0
    return shape, rows, D, code, w_code, stride, dev


def kda_rmsnorm_fwd(x, weight, residual=None, *, eps=1e-6, output_rstd=False, out=None, residual_out=None):
    """RMS norm over the last axis of h = x + residual (x alone without one). Returns
    ``(y, h or None, rstd or None)``: y = h (mean h^2 + eps)^-1/2 weight and h in x's dtype
    (h only with a residual), rstd float32 [...] with ``output_rstd`` (the backward's
    input). ``out`` and ``residual_out`` may each be ``residual`` or, where it is contiguous,
    ``x``, but not the same one."""
    lib = _load()
    shape, rows, D, code, w_code, stride, dev = _norm_inputs(x, weight, residual)
    if out is None:
        out = x.new_empty(shape)
    else:
        _want("out", out, shape, (x.dtype,), dev)
        _apart("out", out, _norm_reads(x, rows, stride, weight, residual), same=("x", "residual"))
    h = _sum_buffer(shape, x, rows, stride, weight, residual, residual_out, dev, out=out)
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=dev) if output_rstd else None
    _call(dev, lib.kda_rmsnorm_fwd, _at(x), stride, _at(weight), _at(residual), _at(out), _at(h), _at(rstd), rows, D,
          eps, code, w_code)
    return out, h, rstd


def _norm_reads(x, rows, stride, weight, residual):
    return (("x", x, rows, stride), *_whole(weight=weight, residual=residual))


def _sum_buffer(shape, x, rows, stride, weight, residual, residual_out, dev, **outputs):
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out belongs to a residual")
        return None
    if residual_out is None:
        return x.new_empty(shape)
    _want("residual_out", residual_out, shape, (x.dtype,), dev)
    _apart("residual_out", residual_out, _norm_reads(x, rows, stride, weight, residual) + _whole(**outputs), same=("x", "residual"))
    return residual_out


def kda_rmsnorm_quant_fwd(x, weight, residual=None, *, eps=1e-6, group=0, out=None, scales=None, residual_out=None):
    """``kda_rmsnorm_fwd`` with an 8-bit output for the projections after it. Returns
    ``(q, scales, h or None)``: q float8_e4m3fn [..., D] and scales float32 with
    y ~ q * scales, one scale for a row (``group`` 0: scales [..., 1]) or for each 128
    columns of it (``group`` 128: [..., D / 128]): s = max(max |y|, 2^-110) / 448."""
    lib = _load()
    if group not in (0, 128):
        raise ValueError(f"group must be 0 (a row) or 128 columns, got {group}")
    shape, rows, D, code, w_code, stride, dev = _norm_inputs(x, weight, residual)
    if group and D % group:
        raise ValueError(f"scales for 128 columns need D a multiple of 128, got {D}")
    sshape = shape[:-1] + ((D // group if group else 1),)
    if out is None:
        out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
    else:
        _want("out", out, shape, (torch.float8_e4m3fn,), dev)
        _apart("out", out, _norm_reads(x, rows, stride, weight, residual))
    if scales is None:
        scales = torch.empty(sshape, dtype=torch.float32, device=dev)
    else:
        _want("scales", scales, sshape, _F32, dev)
        _apart("scales", scales, _norm_reads(x, rows, stride, weight, residual) + _whole(out=out))
    h = _sum_buffer(shape, x, rows, stride, weight, residual, residual_out, dev, out=out, scales=scales)
    _call(dev, lib.kda_rmsnorm_quant_fwd, _at(x), stride, _at(weight), _at(residual), _at(out), _at(scales), _at(h),
          rows, D, group or D, eps, code, w_code)
    return out, scales, h


def kda_rmsnorm_bwd_workspace_bytes(rows, D, dtype=KDA_BF16) -> int:
    if isinstance(dtype, torch.dtype):
        dtype = _CODES[dtype]
    return int(_load().kda_rmsnorm_bwd_workspace_bytes(rows, D, int(dtype)))


def kda_rmsnorm_bwd(dy, h, weight, rstd, dh=None, *, workspace=None):
    """Gradients of ``kda_rmsnorm_fwd`` from its h (x without a residual) and rstd. ``dh``:
    the gradient that reaches h along the residual stream, or None. Returns
    ``(dx, dweight)``: dx in h's dtype is the gradient of x and of the residual alike,
    dweight float32 [D]."""
    lib = _load()
    shape, rows, D, code, w_code, _, dev = _norm_inputs(h, weight, dh)
    _want("h", h, shape, _FLOAT, dev)
    _want("dy", dy, shape, (h.dtype,), dev)
    _want("rstd", rstd, shape[:-1], _F32, dev)
    dx = h.new_empty(shape)
    dweight = torch.empty(D, dtype=torch.float32, device=dev)
    if workspace is not None:
        _apart("workspace", workspace, _whole(dy=dy, h=h, weight=weight, rstd=rstd, dh=dh))
    workspace = _bytes("workspace", workspace, lib.kda_rmsnorm_bwd_workspace_bytes(rows, D, code), dev)
    _call(dev, lib.kda_rmsnorm_bwd, _at(dy), _at(h), _at(weight), _at(rstd), _at(dh), _at(dx), _at(dweight), rows, D,
          code, w_code, _at(workspace), _size(workspace))
    return dx, dweight
