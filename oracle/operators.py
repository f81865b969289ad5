"""fp64 oracle of the gated linear recurrence, layer norm and the state moves,
written from their definitions with numpy, token by token and row by row."""
from __future__ import annotations

import numpy as np


def _spans(B, T, cu):
    if cu is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    return list(zip(cu[:-1], cu[1:]))


def scan(x, log_alpha, init=None, cu=None):
    """h_t = exp(log_alpha_t) h_{t-1} + x_t; x [B,T,D].  Returns (h, final [N,D])."""
    B, T, D = x.shape
    xs, a = x.reshape(-1, D).astype(np.float64), np.exp(log_alpha.reshape(-1, D).astype(np.float64))
    spans = _spans(B, T, cu)
    h, final = np.zeros_like(xs), np.zeros((len(spans), D))
    for n, (t0, t1) in enumerate(spans):
        s = np.zeros(D) if init is None else init[n].astype(np.float64)
        for t in range(t0, t1):
            s = a[t] * s + xs[t]
            h[t] = s
        final[n] = s
    return h.reshape(x.shape), final


def scan_bwd(log_alpha, h, d_h, init=None, d_final=None, cu=None):
    """Gradients of scan with h given: (dx, dlog_alpha, d_init)."""
    B, T, D = h.shape
    hs, a = h.reshape(-1, D).astype(np.float64), np.exp(log_alpha.reshape(-1, D).astype(np.float64))
    dh = d_h.reshape(-1, D).astype(np.float64)
    spans = _spans(B, T, cu)
    dx, dl, d_init = np.zeros_like(hs), np.zeros_like(hs), np.zeros((len(spans), D))
    for n, (t0, t1) in enumerate(spans):
        e = np.zeros(D) if d_final is None else d_final[n].astype(np.float64)
        s0 = np.zeros(D) if init is None else init[n].astype(np.float64)
        for t in range(t1 - 1, t0 - 1, -1):
            dx[t] = dh[t] + e
            e = a[t] * dx[t]
            dl[t] = e * (hs[t - 1] if t > t0 else s0)
        d_init[n] = e
    return dx.reshape(h.shape), dl.reshape(h.shape), d_init


def layernorm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last axis of x [R, D]."""
    x = x.astype(np.float64)
    mean = x.sum(1) / x.shape[1]
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).sum(1) / x.shape[1] + eps)
    y = c * rstd[:, None]
    if weight is not None:
        y = y * weight.astype(np.float64)
    if bias is not None:
        y = y + bias.astype(np.float64)
    return y, mean, rstd


def layernorm_bwd(dy, x, mean, rstd, weight=None):
    """(dx, dweight, dbias) with the statistics as given."""
    dy, x, mean, rstd = (v.astype(np.float64) for v in (dy, x, mean, rstd))
    xh = (x - mean[:, None]) * rstd[:, None]
    u = dy if weight is None else dy * weight.astype(np.float64)
    D = x.shape[1]
    dx = rstd[:, None] * (u - u.sum(1, keepdims=True) / D - xh * (u * xh).sum(1, keepdims=True) / D)
    return dx, (dy * xh).sum(0), dy.sum(0)


def state_move(state, src, dst):
    """state [L, P, ...]: new[:, dst] = old[:, src], zeros for src = -1."""
    new = state.copy()
    for a, b in zip(src, dst):
        new[:, b] = state[:, a] if a >= 0 else 0
    return new
