"""Pins of the layer oracle (CPU): its gradients against central differences of its forwards, its
forwards against forms written another way."""
import numpy as np
import pytest

import oracle
from oracle import layer as L

CU = np.array([0, 3, 3, 4, 9])


def _rand(rng, *shape):
    return rng.standard_normal(shape)


def _difference(f, v, h=1e-6):
    """The gradient of the scalar function f at v by central differences."""
    g = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        keep = v[i]
        v[i] = keep + h
        up = f()
        v[i] = keep - h
        down = f()
        v[i] = keep
        g[i] = (up - down) / (2 * h)
    return g


# Central differences of an O(1) sum in fp64 with h = 1e-6: rounding 1e-16 / 1e-6 = 1e-10 per unit of the
# sum (about 50 here), truncation h^2 = 1e-12.
TOL = dict(atol=2e-8, rtol=1e-6)


def _ssm_case(soft, gate, start, groups):
    rng = np.random.default_rng(7)
    T, ch, n = 9, 4, 3
    return dict(x=_rand(rng, T, ch), dt=0.3 * _rand(rng, T, ch) + (0 if soft else 0.5), B=_rand(rng, T, groups, n),
                C=_rand(rng, T, groups, n), A=-np.exp(_rand(rng, ch, n)), S0=_rand(rng, 4, ch, n) if start else None,
                cu=CU, D=_rand(rng, ch), dt_bias=0.2 * _rand(rng, ch), z=_rand(rng, T, ch) if gate else None,
                soft=soft), _rand(rng, T, ch), _rand(rng, 4, ch, n)


@pytest.mark.parametrize("soft,gate,start,groups", [(True, True, True, 2), (False, False, False, 1), (True, False, True, 4)])
def test_ssm_backward_differences(soft, gate, start, groups):
    k, dy, dS_T = _ssm_case(soft, gate, start, groups)

    def loss():
        y, S = L.ssm(**k)
        return float((y * dy).sum() + (S * dS_T).sum())

    g = L.ssm_backward(dy=dy, dS_T=dS_T, **k)
    for name in ("x", "dt", "B", "C", "A", "D", "dt_bias", "z", "S0"):
        if k[name] is not None:
            np.testing.assert_allclose(g["d" + name], _difference(loss, k[name]), err_msg=name, **TOL)


def test_ssm_is_a_scalar_gate_recurrence():
    """One decay per channel and no read-back: with A the same for every state the scan of a channel is the
    gated outer-product recurrence S = alpha S + (delta x) B, read by C."""
    k, _, _ = _ssm_case(True, False, True, 1)
    k["A"] = np.repeat(k["A"][:, :1], 3, axis=1)
    y, S_T = L.ssm(**k)
    delta = np.log1p(np.exp(k["dt"] + k["dt_bias"]))
    for s in range(4):
        S = k["S0"][s].copy()
        for t in range(CU[s], CU[s + 1]):
            S = np.diag(np.exp(delta[t] * k["A"][:, 0])) @ S + np.outer(delta[t] * k["x"][t], k["B"][t, 0])
            np.testing.assert_allclose(y[t], S @ k["C"][t, 0] + k["D"] * k["x"][t], rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(S_T[s], S, rtol=1e-12, atol=1e-12)


def test_ssm_states_and_continuation():
    k, _, _ = _ssm_case(True, True, True, 2)
    y, S_T = L.ssm(**k)
    before = L.ssm_states(**k)
    np.testing.assert_array_equal(before[0], k["S0"][0])
    # the last sequence cut at token 6, continued from the state before it
    cut = dict(k, **{n: k[n][6:9] for n in ("x", "dt", "B", "C", "z")}, S0=before[6:7], cu=None)
    y2, S2 = L.ssm(**cut)
    np.testing.assert_allclose(y2, y[6:9], rtol=1e-13)
    np.testing.assert_allclose(S2[0], S_T[3], rtol=1e-13)
    np.testing.assert_array_equal(S_T[1], k["S0"][1])  # a sequence without tokens


@pytest.mark.parametrize("W,bias,state", [(4, True, True), (1, True, False), (2, False, True), (8, True, True)])
def test_conv_and_backward(W, bias, state):
    rng = np.random.default_rng(W)
    x, w, dy = _rand(rng, 9, 3), _rand(rng, 3, W), _rand(rng, 9, 3)
    b, st = _rand(rng, 3) if bias else None, _rand(rng, 4, W - 1, 3) if state else None
    y, last = L.conv(x, w, CU, st, b)
    if not bias:
        y_ref, last_ref = oracle.short_conv_swish(x, w, CU, st)
        np.testing.assert_allclose(y, y_ref, rtol=1e-13)
        np.testing.assert_array_equal(last, last_ref)
    dx, dw, db, dstate = L.conv_backward(x, w, dy, CU, st, b)
    loss = lambda: float((L.conv(x, w, CU, st, b)[0] * dy).sum())
    for got, v in ((dx, x), (dw, w)) + (((db, b),) if bias else ()) + (((dstate, st),) if state else ()):
        np.testing.assert_allclose(got, _difference(loss, v), **TOL)


@pytest.mark.parametrize("post,gate,scale,pre,res", [(1, 1, 1, 1, 1), (0, 0, 0, 1, 1), (1, 0, 1, 1, 0), (0, 1, 0, 1, 1),
                                                     (1, 1, 1, 0, 1)])
def test_norm_backward_differences(post, gate, scale, pre, res):
    rng = np.random.default_rng(11)
    pick = lambda has, *shape: _rand(rng, *shape) if has else None
    k = dict(y=_rand(rng, 4, 6), r=pick(res, 4, 6), w_pre=pick(pre, 6), w_post=pick(post, 6), gate=pick(gate, 4, 6),
             scale=pick(scale, 6), res_scale=0.7, eps=1e-3)
    dx, dr = pick(pre, 4, 6), _rand(rng, 4, 6)

    def loss():
        x, out = L.norm(**k)
        return float((out * dr).sum() + (0 if x is None else (x * dx).sum()))

    g = L.norm_backward(dx=dx, dr=dr, **k)
    for name in ("y", "r", "w_pre", "w_post", "gate", "scale"):
        if k[name] is not None:
            np.testing.assert_allclose(g["d" + name], _difference(loss, k[name]), err_msg=name, **TOL)


def test_norm_by_hand():
    x, out = L.norm(np.array([[3.0, 4.0]]), np.array([[1.0, 0.0]]), np.array([1.0, 2.0]), np.array([2.0, 1.0]),
                    np.array([[0.0, np.log(3.0)]]), np.array([1.0, 0.5]), 2.0, 0.0)
    u = np.array([6.0, 4.0]) / np.sqrt(12.5) * np.array([0.5, 0.75]) * np.array([1.0, 0.5])
    np.testing.assert_allclose(out[0], np.array([2.0, 0.0]) + u, rtol=1e-14)
    np.testing.assert_allclose(x[0], out[0] / np.sqrt((out[0] ** 2).mean()) * np.array([1.0, 2.0]), rtol=1e-14)
