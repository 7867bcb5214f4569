"""fp64 CPU oracle for the layer around the recurrences -- TEST INFRASTRUCTURE (numpy only).

* :func:`ssm` / :func:`ssm_backward` -- the selective state space scan token by token, and the
  gradients of its outputs by reverse-mode differentiation of that loop;
* :func:`conv` / :func:`conv_backward` -- the causal short convolution with a bias, then Swish;
* :func:`norm` / :func:`norm_backward` -- the norm after a block, its gate and residual scale, the
  residual stream, and the norm before the next block.

The backward functions are pinned to central differences of the forward ones in the CPU tests.
Arrays are numpy (any real dtype, converted to fp64); packed axes as in the package.
"""
from __future__ import annotations

import numpy as np


def _f64(v):
    return None if v is None else np.asarray(v, dtype=np.float64)


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def _bounds(cu, T):
    cu = np.array([0, T]) if cu is None else np.asarray(cu, dtype=np.int64)
    return [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def _ssm_inputs(x, dt, B, C, A, S0, cu, D, dt_bias, z, soft):
    x, dt, B, C, A, S0, D, dt_bias, z = map(_f64, (x, dt, B, C, A, S0, D, dt_bias, z))
    T, ch = x.shape
    per = ch // B.shape[1]
    Bd, Cd = np.repeat(B, per, axis=1), np.repeat(C, per, axis=1)  # [T, channels, states]
    raw = dt if dt_bias is None else dt + dt_bias
    delta = softplus(raw) if soft else raw
    seqs = _bounds(cu, T)
    S0 = np.zeros((len(seqs), ch, A.shape[1])) if S0 is None else S0
    return x, Bd, Cd, A, S0, (np.zeros(ch) if D is None else D), z, raw, delta, seqs


def ssm(x, dt, B, C, A, S0=None, cu=None, D=None, dt_bias=None, z=None, soft=True):
    """(y [T, channels], S_T [N, channels, states])."""
    x, Bd, Cd, A, S0, D, z, _, delta, seqs = _ssm_inputs(x, dt, B, C, A, S0, cu, D, dt_bias, z, soft)
    y, S_T = np.zeros_like(x), S0.copy()
    for s, (b, e) in enumerate(seqs):
        h = S0[s]
        for t in range(b, e):
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * Bd[t]
            y[t] = (Cd[t] * h).sum(-1) + D * x[t]
        S_T[s] = h
    if z is not None:
        y = y * z * sigmoid(z)
    return y, S_T


def ssm_states(x, dt, B, C, A, S0=None, cu=None, D=None, dt_bias=None, z=None, soft=True):
    """[T, channels, states]: the state before each token."""
    x, Bd, Cd, A, S0, D, z, _, delta, seqs = _ssm_inputs(x, dt, B, C, A, S0, cu, D, dt_bias, z, soft)
    out = np.zeros((x.shape[0],) + A.shape)
    for s, (b, e) in enumerate(seqs):
        h = S0[s]
        for t in range(b, e):
            out[t] = h
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * x[t])[:, None] * Bd[t]
    return out


def ssm_backward(x, dt, B, C, A, dy, dS_T=None, S0=None, cu=None, D=None, dt_bias=None, z=None, soft=True):
    """Gradients of <dy, y> + <dS_T, S_T>: a dict with dx, ddt, dB, dC, dz, dA, dD, ddt_bias, dS0."""
    groups, per = np.shape(B)[1], np.shape(x)[1] // np.shape(B)[1]
    x, Bd, Cd, A, S0, D, z, raw, delta, seqs = _ssm_inputs(x, dt, B, C, A, S0, cu, D, dt_bias, z, soft)
    dy, dS_T = _f64(dy), _f64(dS_T)
    T, ch = x.shape
    n = A.shape[1]
    g = dict(dx=np.zeros_like(x), ddt=np.zeros_like(x), dz=None if z is None else np.zeros_like(x),
             dA=np.zeros_like(A), dD=np.zeros(ch), ddt_bias=np.zeros(ch),
             dS0=np.zeros_like(S0) if dS_T is None else dS_T.copy())
    dBd, dCd = np.zeros((T, ch, n)), np.zeros((T, ch, n))
    for s, (b, e) in enumerate(seqs):
        hs = [S0[s]]
        for t in range(b, e):
            hs.append(np.exp(delta[t][:, None] * A) * hs[-1] + (delta[t] * x[t])[:, None] * Bd[t])
        G = g["dS0"][s].copy()  # dS_T, or zero: the gradient of the state after the last token
        for t in range(e - 1, b - 1, -1):
            h, before = hs[t - b + 1], hs[t - b]
            gy = dy[t]
            if z is not None:
                sg = sigmoid(z[t])
                g["dz"][t] = gy * ((Cd[t] * h).sum(-1) + D * x[t]) * sg * (1 + z[t] * (1 - sg))
                gy = gy * z[t] * sg
            G = G + Cd[t] * gy[:, None]
            dCd[t] = h * gy[:, None]
            a = np.exp(delta[t][:, None] * A)
            dBd[t] = G * (delta[t] * x[t])[:, None]
            gb = (G * Bd[t]).sum(-1)
            g["dx"][t] = delta[t] * gb + D * gy
            g["dD"] += gy * x[t]
            ga = G * before * a  # gradient of delta A
            g["dA"] += ga * delta[t][:, None]
            gd = (ga * A).sum(-1) + gb * x[t]
            g["ddt"][t] = gd * sigmoid(raw[t]) if soft else gd
            G = G * a
        g["dS0"][s] = G
    g["ddt_bias"] = g["ddt"].sum(0)
    g["dB"] = dBd.reshape(T, groups, per, n).sum(2)
    g["dC"] = dCd.reshape(T, groups, per, n).sum(2)
    return g


def _windows(x, W, cu, state):
    """Per sequence: its rows with the W - 1 rows before them."""
    for s, (b, e) in enumerate(_bounds(cu, x.shape[0])):
        before = np.zeros((W - 1, x.shape[1])) if state is None else state[s]
        yield s, b, e, np.concatenate([before, x[b:e]])


def conv(x, w, cu=None, state=None, bias=None):
    """(y [T, C], last W - 1 raw inputs of each sequence [N, W-1, C])."""
    x, w, state, bias = map(_f64, (x, w, state, bias))
    W, y, last = w.shape[1], np.zeros_like(x), []
    for s, b, e, rows in _windows(x, W, cu, state):
        v = np.zeros((e - b, x.shape[1])) if bias is None else np.tile(bias, (e - b, 1))
        for j in range(W):
            v = v + w[:, j] * rows[j:j + e - b]
        y[b:e] = v * sigmoid(v)
        last.append(rows[e - b:])
    return y, np.stack(last)


def conv_backward(x, w, dy, cu=None, state=None, bias=None):
    """(dx [T, C], dw [C, W], dbias [C], dstate [N, W-1, C]) of <dy, y>."""
    x, w, dy, state, bias = map(_f64, (x, w, dy, state, bias))
    W = w.shape[1]
    dx, dw, db, dstate = np.zeros_like(x), np.zeros_like(w), np.zeros(x.shape[1]), []
    for s, b, e, rows in _windows(x, W, cu, state):
        L = e - b
        v = np.zeros((L, x.shape[1])) if bias is None else np.tile(bias, (L, 1))
        for j in range(W):
            v = v + w[:, j] * rows[j:j + L]
        sg = sigmoid(v)
        g = dy[b:e] * sg * (1 + v * (1 - sg))
        drows = np.zeros_like(rows)
        for j in range(W):
            drows[j:j + L] += g * w[:, j]
            dw[:, j] += (g * rows[j:j + L]).sum(0)
        db += g.sum(0)
        dx[b:e] = drows[W - 1:]
        dstate.append(drows[:W - 1])
    return dx, dw, db, np.stack(dstate)


def norm(y, r, w_pre, w_post=None, gate=None, scale=None, res_scale=1.0, eps=1e-6):
    """(x, r'): r' = res_scale r + scale sigmoid(gate) RMSNorm(y) w_post, x = RMSNorm(r') w_pre."""
    y, r, w_pre, w_post, gate, scale = map(_f64, (y, r, w_pre, w_post, gate, scale))
    u = y if w_post is None else y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w_post
    u = u if gate is None else u * sigmoid(gate)
    u = u if scale is None else u * scale
    out = u if r is None else res_scale * r + u
    x = None if w_pre is None else out / np.sqrt((out * out).mean(-1, keepdims=True) + eps) * w_pre
    return x, out


def norm_backward(y, r, w_pre, dx, dr=None, w_post=None, gate=None, scale=None, res_scale=1.0, eps=1e-6):
    """Gradients of <dx, x> + <dr, r'>: a dict with dy, dr, dgate, dw_post, dscale, dw_pre."""
    y, r, w_pre, dx, dr, w_post, gate, scale = map(_f64, (y, r, w_pre, dx, dr, w_post, gate, scale))
    _, out = norm(y, r, w_pre, w_post, gate, scale, res_scale, eps)
    g = dict.fromkeys(("dgate", "dw_post", "dscale", "dw_pre"))
    d = np.zeros_like(out) if dr is None else dr.copy()
    if w_pre is not None:
        rs = 1 / np.sqrt((out * out).mean(-1, keepdims=True) + eps)
        hat = out * rs
        g["dw_pre"] = (dx * hat).sum(0)
        dh = dx * w_pre
        d = d + rs * (dh - hat * (dh * hat).mean(-1, keepdims=True))
    g["dr"] = res_scale * d
    rs = None if w_post is None else 1 / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
    u = y if rs is None else y * rs * w_post
    m = 1.0 if gate is None else sigmoid(gate)
    if scale is not None:
        g["dscale"] = (d * m * u).sum(0)
        d = d * scale
    if gate is not None:
        g["dgate"] = d * u * m * (1 - m)
        d = d * m
    if rs is not None:
        hat = y * rs
        g["dw_post"] = (d * hat).sum(0)
        dh = d * w_post
        d = rs * (dh - hat * (dh * hat).mean(-1, keepdims=True))
    g["dy"] = d
    return g
