"""The fp64 oracle of the operators around the mixer against closed forms, scalar brute
force and finite differences (CPU)."""
import math

import numpy as np
import pytest

from oracle import layer


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_is_the_scalar_sum(W):
    r = rng(W)
    seqs = [(0, 3), (3, 0), (3, 1), (4, 5)]
    x, w, b = r.normal(size=(9, 2)), r.normal(size=(2, W)), r.normal(size=2)
    state = r.normal(size=(4, W - 1, 2))
    y, final, _ = layer.conv_fwd(x, w, b, state, seqs, True)
    for n, (at, ln) in enumerate(seqs):
        seen = [list(v) for v in state[n]] + [list(v) for v in x[at:at + ln]]
        for t in range(ln):
            for d in range(2):
                pre = b[d] + sum(w[d, i] * seen[t + i][d] for i in range(W))
                assert math.isclose(y[at + t, d], pre / (1 + math.exp(-pre)), rel_tol=1e-12)
        assert np.array_equal(final[n], np.array(seen[ln:]))


def test_conv_of_a_delta_gives_the_taps():
    x = np.zeros((6, 1))
    x[1] = 1.0
    y, _, _ = layer.conv_fwd(x, np.array([[1.0, 2.0, 3.0, 4.0]]), None, None, [(0, 6)], False)
    assert y[:, 0].tolist() == [0, 4, 3, 2, 1, 0]


@pytest.mark.parametrize("silu", [False, True])
def test_conv_gradients_are_the_differences(silu):
    r = rng(7)
    seqs = [(0, 4), (4, 0), (4, 1), (5, 2)]
    W, D, rows = 4, 2, 7
    x, w, b = r.normal(size=(rows, D)), r.normal(size=(D, W)), r.normal(size=D)
    state, dy, df = r.normal(size=(4, W - 1, D)), r.normal(size=(rows, D)), r.normal(size=(4, W - 1, D))
    got = layer.conv_bwd(dy, x, w, b, state, df, seqs, silu)

    def value():
        y, f, _ = layer.conv_fwd(x, w, b, state, seqs, silu)
        return (y * dy).sum() + (f * df).sum()

    for g, v in zip(got[:4], (x, w, b, state)):
        for i in np.ndindex(v.shape):
            old, h = v[i], 1e-6
            v[i] = old + h
            up = value()
            v[i] = old - h
            down = value()
            v[i] = old
            assert math.isclose(g[i], (up - down) / (2 * h), rel_tol=1e-6, abs_tol=1e-7)


def test_ssm_closed_forms():
    r = rng(3)
    K, V, T = 2, 3, 5
    x, b, c = r.normal(size=(T, 1, V)), r.normal(size=(T, 1, K)), r.normal(size=(T, 1, K))
    dt = np.abs(r.normal(size=(T, 1)))
    A_log, h0 = np.array([0.3]), r.normal(size=(1, 1, K, V))
    y, final, _, _ = layer.ssm(x, dt, A_log, b, c, np.array([0.7]), None, h0, [(0, T)], False)
    a = -math.exp(0.3)
    for t in range(T):
        S = h0[0, 0] * math.exp(a * dt[:t + 1, 0].sum())
        for j in range(t + 1):
            S = S + math.exp(a * dt[j + 1:t + 1, 0].sum()) * dt[j, 0] * np.outer(b[j, 0], x[j, 0])
        assert np.allclose(y[t, 0], c[t, 0] @ S + 0.7 * x[t, 0], rtol=1e-12)
    assert np.allclose(final[0, 0], S, rtol=1e-12)


def test_ssm_heads_groups_sequences_and_softplus():
    r = rng(4)
    HV, H, K, V = 4, 2, 2, 2
    seqs = [(0, 2), (2, 0), (2, 3)]
    x, dt = r.normal(size=(6, HV, V)), r.normal(size=(6, HV))
    b, c = r.normal(size=(6, H, K)), r.normal(size=(6, H, K))
    A, bias, h0 = r.normal(size=HV), r.normal(size=HV), r.normal(size=(3, HV, K, V))
    y, final, _, _ = layer.ssm(x, dt, A, b, c, None, bias, h0, seqs, True)
    assert np.isnan(y[5]).all() and np.array_equal(final[1], h0[1])
    for n, (at, ln) in enumerate(seqs):
        for hv in range(HV):
            one = layer.ssm(x[at:at + ln, hv:hv + 1], np.log1p(np.exp(dt[at:at + ln, hv:hv + 1] + bias[hv])), A[hv:hv + 1],
                            b[at:at + ln, hv // 2:hv // 2 + 1], c[at:at + ln, hv // 2:hv // 2 + 1], None, None,
                            h0[n:n + 1, hv:hv + 1], [(0, ln)], False)
            assert np.allclose(one[0][:, 0], y[at:at + ln, hv], rtol=1e-12)
            assert np.allclose(one[1][0, 0], final[n, hv], rtol=1e-12)


def test_rmsnorm_rows_and_scales():
    y, h, r = layer.rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), np.array([[0.0, 0.0]]), 0.0)
    root = math.sqrt(12.5)
    assert np.allclose(y, [[3 / root, 8 / root]]) and np.allclose(r, [1 / root])
    assert np.allclose(layer.fp8_scales(np.array([[1.0, -448.0, 2.0, 0.0], [0, 0, 0, 0]]), 2),
                       [[1.0, 2 / 448], [2.0 ** -110 / 448] * 2])


def test_rmsnorm_gradients_are_the_differences():
    r = rng(9)
    h, w, dy, dh = r.normal(size=(3, 5)), r.normal(size=5), r.normal(size=(3, 5)), r.normal(size=(3, 5))
    dx, dw = layer.rmsnorm_bwd(dy, h, w, layer.rmsnorm(h, w, None, 1e-3)[2], dh)

    def value():
        return (layer.rmsnorm(h, w, None, 1e-3)[0] * dy).sum() + (h * dh).sum()

    for g, v in ((dx, h), (dw, w)):
        for i in np.ndindex(v.shape):
            old, e = v[i], 1e-6
            v[i] = old + e
            up = value()
            v[i] = old - e
            down = value()
            v[i] = old
            assert math.isclose(g[i], (up - down) / (2 * e), rel_tol=1e-6, abs_tol=1e-7)


def planted(name):
    """Copies of the oracle's functions with one mistake each, which the checks above must see."""
    src = open(layer.__file__).read()
    old, new, check = {
        "taps reversed": ("ext[t:t + W] * w.T\n            pre", "ext[t:t + W] * w.T[::-1]\n            pre", test_conv_of_a_delta_gives_the_taps),
        "state of the first rows": ("final[n] = ext[ln:]", "final[n] = ext[:W - 1]", lambda: test_conv_is_the_scalar_sum(4)),
        "silu's slope without its second term": ("d * s * (1 + pre * (1 - s))", "d * s", lambda: test_conv_gradients_are_the_differences(True)),
        "final state's gradient dropped": ("grad[ln:] += f(dfinal[n])", "pass", lambda: test_conv_gradients_are_the_differences(False)),
        "read before the write": ('y[t] = np.einsum("hk,hkv->hv", f(c[t][head]), S)', 'y[t] = np.einsum("hk,hkv->hv", f(c[t][head]), S - f(b[t][head])[:, :, None] * f(step[:, None] * x[t])[:, None, :])', test_ssm_closed_forms),
        "decay of A_log itself": ("np.exp(-np.exp(A_log) * step)", "np.exp(-A_log * step)", test_ssm_closed_forms),
        "groups taken in turn": ("np.arange(HV) // (HV // H)", "np.arange(HV) % H", test_ssm_heads_groups_sequences_and_softplus),
        "the mean's gradient dropped": ("(g - xh * np.mean(g * xh, -1, keepdims=True))", "g", test_rmsnorm_gradients_are_the_differences),
        "sum for mean": ("np.sqrt(np.mean(h * h, -1) + eps)", "np.sqrt(np.sum(h * h, -1) + eps)", test_rmsnorm_rows_and_scales),
    }[name]
    assert src.count(old) == 1, name
    ns = {}
    exec(compile(src.replace(old, new), "planted", "exec"), ns)
    return ns, check


@pytest.mark.parametrize("name", ["taps reversed", "state of the first rows", "silu's slope without its second term",
                                  "final state's gradient dropped", "read before the write", "decay of A_log itself",
                                  "groups taken in turn", "the mean's gradient dropped", "sum for mean"])
def test_planted_mistakes_are_seen(name, monkeypatch):
    ns, check = planted(name)
    for f in ("conv_fwd", "conv_bwd", "ssm", "rmsnorm", "rmsnorm_bwd", "fp8_scales"):
        monkeypatch.setattr(layer, f, ns[f])
    with pytest.raises(AssertionError):
        check()
