"""The operators around the mixer in fp64 numpy, written out token by token: the short
causal convolution and its gradients, the selective state space scan, the RMS norm, its
gradients and its 8-bit output. Test infrastructure only; shares nothing with the HIP path.

Sequences are (first row, length) pairs over the flattened rows; rows outside every
sequence come back as NaN."""
import numpy as np


def spans(B, T, cu=None):
    if cu is None:
        return [(b * T, T) for b in range(B)]
    return [(int(a), int(b) - int(a)) for a, b in zip(cu[:-1], cu[1:])]


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def conv_fwd(x, w, bias, state, seqs, silu):
    """x [rows, D], w [D, W], bias [D] or None, state [N, W-1, D] or None -> y, final, |terms|
    (the sum of the magnitudes behind each pre-activation)."""
    rows, D = x.shape
    W = w.shape[1]
    y, mag = np.full((rows, D), np.nan), np.full((rows, D), np.nan)
    final = np.zeros((len(seqs), W - 1, D))
    b = np.zeros(D) if bias is None else bias
    for n, (at, ln) in enumerate(seqs):
        before = np.zeros((W - 1, D)) if state is None else state[n]
        ext = np.concatenate([before, x[at:at + ln]])
        for t in range(ln):
            terms = ext[t:t + W] * w.T
            pre = b + terms.sum(0)
            y[at + t] = pre * sigmoid(pre) if silu else pre
            mag[at + t] = np.abs(b) + np.abs(terms).sum(0)
        final[n] = ext[ln:]
    return y, final, mag


def conv_bwd(dy, x, w, bias, state, dfinal, seqs, silu):
    """-> dx [rows, D], dw [D, W], db [D], dstate [N, W-1, D], and the same from magnitudes."""
    rows, D = x.shape
    W = w.shape[1]
    b = np.zeros(D) if bias is None else bias
    out = []
    for mag in (False, True):
        f = np.abs if mag else (lambda v: v)
        dx, dw, db = np.full((rows, D), np.nan), np.zeros((D, W)), np.zeros(D)
        dstate = np.zeros((len(seqs), W - 1, D))
        for n, (at, ln) in enumerate(seqs):
            before = np.zeros((W - 1, D)) if state is None else state[n]
            ext = np.concatenate([before, x[at:at + ln]])
            grad = np.zeros_like(ext)
            for t in range(ln):
                d = dy[at + t]
                if silu:
                    pre = b + (ext[t:t + W] * w.T).sum(0)
                    s = sigmoid(pre)
                    d = d * s * (f(pre) * (1 - s) + 1) if mag else d * s * (1 + pre * (1 - s))
                d = f(d)
                grad[t:t + W] += d * f(w.T)
                dw += (d * f(ext[t:t + W])).T
                db += d
            if dfinal is not None:
                grad[ln:] += f(dfinal[n])
            dx[at:at + ln] = grad[W - 1:]
            dstate[n] = grad[:W - 1]
        out.append((dx, dw, db, dstate))
    return out[0] + (out[1],)


def softplus(z):
    return np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z)))


def ssm(x, dt, A_log, b, c, D, dt_bias, state, seqs, use_softplus):
    """x [rows, HV, V], dt [rows, HV], b, c [rows, H, K] -> y, final state, and both from
    magnitudes (every product taken as its absolute value)."""
    rows, HV, V = x.shape
    H, K = b.shape[1:]
    head = np.arange(HV) // (HV // H)
    out = []
    for mag in (False, True):
        f = np.abs if mag else (lambda v: v)
        y = np.full((rows, HV, V), np.nan)
        final = np.zeros((len(seqs), HV, K, V))
        for n, (at, ln) in enumerate(seqs):
            S = np.zeros((HV, K, V)) if state is None else f(state[n]).copy()
            for t in range(at, at + ln):
                z = dt[t] + (0 if dt_bias is None else dt_bias)
                step = softplus(z) if use_softplus else z
                S = S * np.exp(-np.exp(A_log) * step)[:, None, None]
                S = S + f(b[t][head])[:, :, None] * f(step[:, None] * x[t])[:, None, :]
                y[t] = np.einsum("hk,hkv->hv", f(c[t][head]), S)
                if D is not None:
                    y[t] += f(D[:, None] * x[t])
            final[n] = S
        out.append((y, final))
    return out[0] + out[1]


def rmsnorm(x, w, res, eps):
    """-> y, h, r"""
    h = x if res is None else x + res
    r = 1.0 / np.sqrt(np.mean(h * h, -1) + eps)
    return h * r[..., None] * w, h, r


def fp8_scales(y, group):
    rows, D = y.shape
    top = np.abs(y.reshape(rows, D // group, group)).max(-1)
    return np.maximum(top, 2.0 ** -110) / 448.0


def rmsnorm_bwd(dy, h, w, r, dh):
    """-> dx, dw"""
    xh = h * r[:, None]
    g = dy * w
    dx = r[:, None] * (g - xh * np.mean(g * xh, -1, keepdims=True))
    return dx + (0 if dh is None else dh), (dy * xh).sum(0)
