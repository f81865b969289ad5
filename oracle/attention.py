"""fp64 oracle of windowed attention with sinks, its gradients and its resident
cache, written from their definitions with numpy, query by query and token by
token."""
from __future__ import annotations

import numpy as np


def visible(p, keys, window, sinks):
    """Indices of the keys 0 .. keys - 1 that the query at position p sees."""
    return [j for j in range(keys) if j <= p and (p - j < window or j < sinks)]


def _sequences(B, T, Tk, cu, cuk):
    if cu is None:
        return [(b * T, (b + 1) * T, b * Tk, (b + 1) * Tk) for b in range(B)]
    return list(zip(cu[:-1], cu[1:], cuk[:-1], cuk[1:]))


def attention(q, k, v, window, sinks=0, cu=None, cuk=None, scale=None):
    """q [B,T,H,d], k, v [B,Tk,KV,d].  Returns (o, lse); a query that sees nothing: 0 and -inf."""
    (B, T, H, d), (_, Tk, KV, _) = q.shape, k.shape
    scale = d ** -0.5 if scale is None else scale
    qs, ks, vs = (x.astype(np.float64).reshape(-1, *x.shape[2:]) for x in (q, k, v))
    o, lse = np.zeros_like(qs), np.full(qs.shape[:2], -np.inf)
    for q0, q1, k0, k1 in _sequences(B, T, Tk, cu, cuk if cuk is not None else cu):
        for i in range(q0, q1):
            see = np.array(visible(i - q0 + (k1 - k0) - (q1 - q0), k1 - k0, window, sinks), dtype=int) + k0
            if not len(see):
                continue
            for h in range(H):
                e = h // (H // KV)
                s = scale * (ks[see, e] @ qs[i, h])
                top = s.max()
                if top == -np.inf:
                    continue
                w = np.exp(s - top)
                lse[i, h] = top + np.log(w.sum())
                o[i, h] = (w / w.sum()) @ vs[see, e]
    return o.reshape(q.shape), lse.reshape(q.shape[:3])


def attention_bwd(d_o, q, k, v, o, lse, window, sinks=0, cu=None, cuk=None, scale=None):
    """Gradients (dq, dk, dv) with o and lse as given."""
    (B, T, H, d), (_, Tk, KV, _) = q.shape, k.shape
    scale = d ** -0.5 if scale is None else scale
    qs, ks, vs, os, gs = (x.astype(np.float64).reshape(-1, *x.shape[2:]) for x in (q, k, v, o, d_o))
    ls = lse.astype(np.float64).reshape(-1, H)
    dq, dk, dv = np.zeros_like(qs), np.zeros_like(ks), np.zeros_like(vs)
    for q0, q1, k0, k1 in _sequences(B, T, Tk, cu, cuk if cuk is not None else cu):
        for i in range(q0, q1):
            see = np.array(visible(i - q0 + (k1 - k0) - (q1 - q0), k1 - k0, window, sinks), dtype=int) + k0
            if not len(see):
                continue
            for h in range(H):
                e = h // (H // KV)
                if ls[i, h] == -np.inf:
                    continue
                p = np.exp(scale * (ks[see, e] @ qs[i, h]) - ls[i, h])
                ds = p * (vs[see, e] @ gs[i, h] - gs[i, h] @ os[i, h])
                dv[see, e] += p[:, None] * gs[i, h]
                dq[i, h] = scale * (ds @ ks[see, e])
                dk[see, e] += scale * ds[:, None] * qs[i, h]
    return dq.reshape(q.shape), dk.reshape(k.shape), dv.reshape(v.shape)


# ---- the resident cache --------------------------------------------------------------

def cache_row(p, window, sinks):
    """The cache row of position p: the sinks' own, then a ring."""
    return p if p < sinks else sinks + (p - sinks) % window


def e4m3(x):
    """A row's values in e4m3 (as the numbers that they stand for, before the scale) and its scale: the least
    power of two 2^e, e >= -126, with max|x| <= 448 * 2^e.  A row that is not finite: NaN throughout."""
    x = np.asarray(x, dtype=np.float64)
    if not np.isfinite(x).all():
        return np.full_like(x, np.nan), np.nan
    e, top = -126, np.abs(x).max()
    while top > 448.0 * 2.0 ** e:
        e += 1
    y = x / 2.0 ** e
    out = np.zeros_like(y)
    for i, value in enumerate(y):
        if value:
            step = 2.0 ** (max(int(np.floor(np.log2(abs(value)))), -6) - 3)
            out[i] = np.round(value / step) * step       # numpy rounds halves to even
    return out, 2.0 ** e


def cache_write(cache, k, v, lengths, sinks, scales=None, slots=None, cu=None):
    """cache [2,P,KV,rows,d] (and scales [2,P,KV,rows], or None) after the tokens of k, v [B,T,KV,d] went in, one
    after the other.  Returns new (cache, scales)."""
    cache, scales = cache.astype(np.float64).copy(), None if scales is None else scales.astype(np.float64).copy()
    window = cache.shape[3] - sinks
    B, T = k.shape[:2]
    cu = [b * T for b in range(B + 1)] if cu is None else cu
    for n in range(len(cu) - 1):
        at = n if slots is None else slots[n]
        if at < 0:
            continue
        for t in range(cu[n], cu[n + 1]):
            row = cache_row(lengths[n] + t - cu[n], window, sinks)
            for side, x in enumerate((k, v)):
                x = x.reshape(-1, *x.shape[2:])
                for h in range(cache.shape[2]):
                    if scales is None:
                        cache[side, at, h, row] = x[t, h]
                    else:
                        cache[side, at, h, row], scales[side, at, h, row] = e4m3(x[t, h])
    return cache, scales


def cache_read(cache, lengths, sinks, scales=None, slots=None):
    """What each sequence's cache holds, in the order of positions: a list of (k, v) [rows, KV, d]."""
    window = cache.shape[3] - sinks
    out = []
    for n, length in enumerate(lengths):
        at = n if slots is None else slots[n]
        if at < 0:
            out.append(None)
            continue
        seen = [*range(min(sinks, length)), *range(max(sinks, length - window), length)]
        rows = [cache_row(p, window, sinks) for p in seen]
        both = []
        for side in range(2):
            x = cache[side, at].astype(np.float64)[:, rows]
            if scales is not None:
                x = x * scales[side, at].astype(np.float64)[:, rows, None]
            both.append(x.transpose(1, 0, 2))
        out.append(tuple(both))
    return out


def step(cache, q, k, v, lengths, sinks, scales=None, slots=None, scale=None):
    """One token of each sequence: (o [N,H,d], new cache, new scales).  Slot -1: nothing is written, o is 0."""
    N, H, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    cache, scales = cache_write(cache, k[:, None], v[:, None], lengths, sinks, scales, slots)
    o = np.zeros(q.shape)
    for n, both in enumerate(cache_read(cache, [x + 1 for x in lengths], sinks, scales, slots)):
        if both is None:
            continue
        for h in range(H):
            e = h // (H // cache.shape[2])
            s = scale * (both[0][:, e] @ q[n, h].astype(np.float64))
            w = np.exp(s - s.max())
            o[n, h] = (w / w.sum()) @ both[1][:, e]
    return o, cache, scales
