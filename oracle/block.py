"""Float64 definitions of the operators of a block, token by token: the gated recurrence a
channel, the short causal convolution and the norms around a block, each with its gradients
written out (pinned by finite differences in the tests). numpy only.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z < 0, e, 1.0) / (1.0 + e)


def _tokens(lens, b, T):
    return T if lens is None else min(max(int(lens[b]), 0), T)


def _gates(f, gate, decay):
    """(a, m) of h = a h + m sigmoid(i) x."""
    with np.errstate(over="ignore"):
        if gate == "log":
            return np.exp(f), np.ones_like(f)
        if gate == "sigmoid":
            return _sigmoid(f), _sigmoid(-f)
    e = -_f64(decay) * _sigmoid(f)
    return np.exp(e), np.sqrt(-np.expm1(2.0 * e))


def scan_forward(x, f, i=None, *, gate="sigmoid", decay=None, h0=None, lens=None, h=None):
    """(h, h_final). x, f, i [B, T, C]; rows of ``h`` behind a length stay."""
    x, f = _f64(x), _f64(f)
    B, T, C = x.shape
    a, m = _gates(f, gate, decay)
    add = m * x * (1.0 if i is None else _sigmoid(_f64(i)))
    state = np.zeros((B, C)) if h0 is None else _f64(h0).copy()
    h = np.zeros((B, T, C)) if h is None else _f64(h).copy()
    for b in range(B):
        for t in range(_tokens(lens, b, T)):
            state[b] = a[b, t] * state[b] + add[b, t]
            h[b, t] = state[b]
    return h, state


def scan_backward(x, f, i=None, *, d_h, gate="sigmoid", decay=None, h0=None, dh_final=None, lens=None):
    """Gradients of sum(h * d_h) + sum(h_final * dh_final): {"dx", "df", "di", "ddecay", "dh0"}
    ("di" with i, "ddecay" for "power")."""
    x, f, d_h = _f64(x), _f64(f), _f64(d_h)
    B, T, C = x.shape
    a, m = _gates(f, gate, decay)
    s = np.ones_like(x) if i is None else _sigmoid(_f64(i))
    sf = _sigmoid(f)
    start = np.zeros((B, C)) if h0 is None else _f64(h0)
    h, _ = scan_forward(x, f, i, gate=gate, decay=decay, h0=h0, lens=lens)
    G = np.zeros((B, C)) if dh_final is None else _f64(dh_final).copy()
    dx, df, di = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    ddecay = np.zeros(C)
    for b in range(B):
        for t in range(_tokens(lens, b, T) - 1, -1, -1):
            lam = G[b] + d_h[b, t]
            before = h[b, t - 1] if t else start[b]
            at, mt, st, xt = a[b, t], m[b, t], s[b, t], x[b, t]
            dx[b, t] = lam * mt * st
            di[b, t] = lam * mt * xt * st * (1.0 - st)
            if gate == "log":
                df[b, t] = lam * before * at
            elif gate == "sigmoid":
                df[b, t] = lam * (before - st * xt) * at * mt
            else:
                # m = sqrt(1 - a^2): d m / d log a = -a^2 / m, taken as 0 where a = 1
                slope = np.divide(at * at, mt, out=np.zeros_like(at), where=mt > 0)
                dlog = lam * (at * before - slope * st * xt)
                df[b, t] = -_f64(decay) * dlog * sf[b, t] * (1.0 - sf[b, t])
                ddecay -= dlog * sf[b, t]
            G[b] = at * lam
    out = {"dx": dx, "df": df, "dh0": G}
    if i is not None:
        out["di"] = di
    if gate == "power":
        out["ddecay"] = ddecay
    return out


def _past(x, W, s0):
    B, _, C = x.shape
    return np.concatenate((np.zeros((B, W - 1, C)) if s0 is None else _f64(s0), x), 1)


def conv_forward(x, w, bias=None, *, activation="silu", s0=None, lens=None, y=None):
    """(y, s_final). x [B, T, C], w [C, W]; rows of ``y`` behind a length stay."""
    x, w = _f64(x), _f64(w)
    B, T, C = x.shape
    W = w.shape[1]
    past = _past(x, W, s0)
    y = np.zeros((B, T, C)) if y is None else _f64(y).copy()
    end = np.zeros((B, W - 1, C))
    for b in range(B):
        n = _tokens(lens, b, T)
        for t in range(n):
            z = (past[b, t:t + W] * w.T).sum(0) + (0.0 if bias is None else _f64(bias))
            y[b, t] = z * _sigmoid(z) if activation == "silu" else z
        end[b] = past[b, n:n + W - 1]
    return y, end


def conv_backward(x, w, bias=None, *, d_y, activation="silu", s0=None, ds_final=None, lens=None):
    """Gradients of sum(y * d_y) + sum(s_final * ds_final): {"dx", "dw", "dbias", "ds0"}."""
    x, w, d_y = _f64(x), _f64(w), _f64(d_y)
    B, T, C = x.shape
    W = w.shape[1]
    past = _past(x, W, s0)
    back = np.zeros_like(past)
    dw, db = np.zeros_like(w), np.zeros(C)
    for b in range(B):
        n = _tokens(lens, b, T)
        for t in range(n):
            dz = d_y[b, t]
            if activation == "silu":
                z = (past[b, t:t + W] * w.T).sum(0) + (0.0 if bias is None else _f64(bias))
                s = _sigmoid(z)
                dz = dz * (s + z * s * (1.0 - s))
            back[b, t:t + W] += dz * w.T
            dw += (dz * past[b, t:t + W]).T
            db += dz
        if ds_final is not None:
            back[b, n:n + W - 1] += _f64(ds_final)[b]
    return {"dx": back[:, W - 1:], "dw": dw, "dbias": db, "ds0": back[:, :W - 1]}


def _rms(x, eps):
    return ((x * x).mean(-1, keepdims=True) + eps) ** -0.5


def _rms_back(x, w, dy, eps):
    """(dx, dw) of x rms(x) w: with r = (mean x^2 + eps)^-1/2, dr/dx = -r^3 x / C."""
    r = _rms(x, eps)
    dn = dy * w
    return r * dn - x * r ** 3 * (dn * x).mean(-1, keepdims=True), (dy * x * r).reshape(-1, x.shape[-1]).sum(0)


def block_norm(residual, y=None, gate=None, *, weight=None, post_norm=False, post_weight=None, scale=None,
               activation="sigmoid", residual_scale=1.0, eps=1e-6, d_residual_out=None, d_out=None):
    """(residual_out, out); with an upstream gradient also {"dr", "dy", "dgate", "dscale",
    "dw_post", "dw"}."""
    r0 = _f64(residual)
    C = r0.shape[-1]
    ones = np.ones(C)
    w, pw, sc = (ones if t is None else _f64(t) for t in (weight, post_weight, scale))
    yv = np.zeros_like(r0) if y is None else _f64(y)
    hat = yv * _rms(yv, eps) if post_norm else yv
    if gate is None:
        act, slope = np.ones_like(r0), np.zeros_like(r0)
    else:
        z = _f64(gate)
        s = _sigmoid(z)
        act, slope = (z * s, s + z * s * (1.0 - s)) if activation == "silu" else (s, s * (1.0 - s))
    u = hat * pw
    r = residual_scale * r0 + sc * act * u
    out = r * _rms(r, eps) * w
    if d_residual_out is None and d_out is None:
        return r, out
    dr = np.zeros_like(r) if d_residual_out is None else _f64(d_residual_out).copy()
    dw = np.zeros(C)
    if d_out is not None:
        back, dw = _rms_back(r, w, _f64(d_out), eps)
        dr = dr + back
    du = dr * sc * act
    rows = lambda t: t.reshape(-1, C).sum(0)  # noqa: E731
    g = {"dr": residual_scale * dr, "dgate": dr * sc * u * slope, "dscale": rows(dr * act * u), "dw": dw}
    if post_norm:
        g["dy"], g["dw_post"] = _rms_back(yv, pw, du, eps)
    else:
        g["dy"], g["dw_post"] = du, np.zeros(C)
    return r, out, g
