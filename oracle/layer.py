"""Float64 definitions of the operators around the delta rule, token by token and row by
row: linear attention with one decay a head and its gradients, the norms of queries and
keys with the position rotation, and the gated norm. numpy only; gradients are written out
and pinned by finite differences in the tests.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def _decay(log_decay):
    return np.exp(_f64(log_decay))[:, None, None]


def linear_forward(q, k, v, log_decay, s0=None, lens=None, o=None):
    """(o, s_final). q, k [B, T, Hk, dk], v [B, T, H, dv]; rows of ``o`` behind a length stay."""
    q, k, v, gam = _f64(q), _f64(k), _f64(v), _decay(log_decay)
    B, T, H, dv = v.shape
    rep = H // k.shape[2]
    S = np.zeros((B, H, k.shape[3], dv)) if s0 is None else _f64(s0).copy()
    o = np.zeros((B, T, H, dv)) if o is None else _f64(o).copy()
    for b in range(B):
        for t in range(T if lens is None else min(max(int(lens[b]), 0), T)):
            S[b] = gam * S[b] + np.repeat(k[b, t], rep, 0)[:, :, None] * v[b, t][:, None, :]
            o[b, t] = (np.repeat(q[b, t], rep, 0)[:, :, None] * S[b]).sum(1)
    return o, S


def linear_backward(q, k, v, log_decay, d_o, s0=None, ds_final=None, lens=None):
    """{"dq", "dk", "dv", "ds0"} of sum(o * d_o) + sum(s_final * ds_final)."""
    q, k, v, d_o, gam = _f64(q), _f64(k), _f64(v), _f64(d_o), _decay(log_decay)
    B, T, H, dv = v.shape
    Hk, dk = k.shape[2:]
    rep = H // Hk
    fold = lambda x: x.reshape(Hk, rep, dk).sum(1)  # noqa: E731
    S = np.zeros((B, H, dk, dv)) if s0 is None else _f64(s0).copy()
    G = np.zeros((B, H, dk, dv)) if ds_final is None else _f64(ds_final).copy()
    out = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v)}
    for b in range(B):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        for t in range(n):
            S[b] = gam * S[b] + np.repeat(k[b, t], rep, 0)[:, :, None] * v[b, t][:, None, :]
            out["dq"][b, t] = fold((S[b] * d_o[b, t][:, None, :]).sum(2))
        for t in range(n - 1, -1, -1):
            G[b] += np.repeat(q[b, t], rep, 0)[:, :, None] * d_o[b, t][:, None, :]
            out["dk"][b, t] = fold((G[b] * v[b, t][:, None, :]).sum(2))
            out["dv"][b, t] = (G[b] * np.repeat(k[b, t], rep, 0)[:, :, None]).sum(1)
            G[b] *= gam
    out["ds0"] = G
    return out


def _rotation(d, rot, positions, cos, sin, interleaved):
    """The rotation of every token as matrices [B, T, d, d]."""
    B, T = positions.shape
    R = np.broadcast_to(np.eye(d), (B, T, d, d)).copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = _f64(cos)[positions, i], _f64(sin)[positions, i]
        R[:, :, a, a], R[:, :, a, b], R[:, :, b, a], R[:, :, b, b] = c, -s, s, c
    return R


def head_norm(x, w=None, *, norm="rms", eps=1e-6, scale=1.0, cos=None, sin=None, positions=None,
              interleaved=False, dy=None):
    """The norm of each head's row, its rotation and its scale; with ``dy`` also the
    gradients: (y, dx, dw)."""
    x = _f64(x)
    B, T, _, d = x.shape
    w = np.ones(d) if w is None else _f64(w)
    count = d if norm == "rms" else 1
    r = ((x * x).sum(-1, keepdims=True) / count + eps) ** -0.5
    pos = np.broadcast_to(np.arange(T), (B, T)) if positions is None else np.asarray(positions, dtype=np.int64)
    rot = 0 if cos is None else 2 * cos.shape[1]
    R = _rotation(d, rot, pos, cos, sin, interleaved)
    n = x * r
    y = np.matmul(R[:, :, None], (n * w)[..., None])[..., 0] * scale
    if dy is None:
        return y
    dz = np.matmul(np.swapaxes(R, -1, -2)[:, :, None], _f64(dy)[..., None])[..., 0] * scale
    dn = dz * w
    # d r / d x = -r^3 x / count
    dx = r * dn - x * r ** 3 / count * (dn * x).sum(-1, keepdims=True)
    return y, dx, (dz * n).sum((0, 1, 2))


def gated_norm(x, gate, w=None, *, eps=1e-6, activation="silu", dy=None):
    """RMS norm of x times act(gate); with ``dy`` also the gradients: (y, dx, dgate, dw)."""
    x, z = _f64(x), _f64(gate)
    d = x.shape[-1]
    w = np.ones(d) if w is None else _f64(w)
    s = 1.0 / (1.0 + np.exp(-z))
    act, slope = (z * s, s + z * s * (1.0 - s)) if activation == "silu" else (s, s * (1.0 - s))
    y = head_norm(x, w, eps=eps) * act
    if dy is None:
        return y
    dy = _f64(dy)
    _, dx, dw = head_norm(x, w, eps=eps, dy=dy * act)
    return y, dx, dy * head_norm(x, w, eps=eps) * slope, dw
