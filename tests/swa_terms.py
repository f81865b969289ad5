"""Gradients of windowed attention in 64 bits, whole matrices at a time, and for each of their elements how far a
result may be from it, by the terms of its own sum.

With u = 2^-24 and h = half a step of the type, for every visible pair (i, j):
  s_ij   a sum of d products in fp32: off by (d + 8) u A_ij, A = scale |q_i| |k_j| element by element;
  P_ij   exp of it less lse, whose product with log2 e is rounded: off by e_ij = (d + 8) u A_ij + 4 u |lse_i| + 16 u, relative;
  dP_ij  a sum of d products: off by (d + 2) u G_ij, G = |d_o_i| |v_j|;     D_i: off by (d + 2) u |d_o_i| |o_i|;
  dS_ij = P (dP - D), rounded to the type as an operand: off by
           x_ij = h |dS_ij| / sqrt 3 + e_ij |dS_ij| + (d + 4) u P_ij G_ij     and P_ij (d + 2) u |d_o_i| |o_i|.
An operand's rounding is at most h, and as its place between two neighbours is as good as random, h / sqrt 3 or less on
average (root mean square).  The terms of an element's sum err independently, so their errors add as squares do: six times
the root of that sum is exceeded once in 10^9.  (A single term's h is below 6 h / sqrt 3 in any case.)  D_i's error is
the same for all of a row's terms: it is added in full.  A sum of n terms in fp32 rounds by sqrt(n) u of the root of the sum
of its squares in the same way.  FP16's subnormal operands: half a step is 2^-25, where the largest |dS| of the sum counts as
2^12 or more: 2^-37 of it each, likewise.
"""
import numpy as np


def _pairs(B, T, Tk, cu, cuk):
    if cu is None:
        return [(b * T, (b + 1) * T, b * Tk, (b + 1) * Tk) for b in range(B)]
    cuk = cu if cuk is None else cuk
    return list(zip(cu[:-1], cu[1:], cuk[:-1], cuk[1:]))


def gradients(do, q, k, v, o, lse, window, sinks=0, cu=None, cuk=None, scale=None, h=0.0):
    """[(gradient, room)] of q, k and v."""
    (B, T, H, d), (_, Tk, KV, _) = q.shape, k.shape
    scale = d ** -0.5 if scale is None else scale
    u, G = 2.0 ** -24, H // KV
    qs, ks, vs, os, gs = (np.asarray(x, dtype=np.float64).reshape(-1, *x.shape[2:]) for x in (q, k, v, o, do))
    ls = lse.reshape(-1, H)
    want = [np.zeros_like(x) for x in (qs, ks, vs)]
    square = [np.zeros_like(x) for x in (qs, ks, vs)]            # of the independent errors
    plain = [np.zeros_like(x) for x in (qs, ks, vs)]             # of the others
    terms = np.zeros(ks.shape)                                   # of a key's sums
    for q0, q1, k0, k1 in _pairs(B, T, Tk, cu, cuk):
        if q1 == q0 or k1 == k0:
            continue
        p, j = np.arange(q1 - q0)[:, None] + (k1 - k0) - (q1 - q0), np.arange(k1 - k0)[None]
        see = (j <= p) & ((p - j < window) | (j < sinks))
        for x in range(H):
            e = x // G
            Q, K, V, O, D = qs[q0:q1, x], ks[k0:k1, e], vs[k0:k1, e], os[q0:q1, x], gs[q0:q1, x]
            L = ls[q0:q1, x][:, None]
            L = np.where(np.isinf(L), np.inf, L)
            P = np.where(see, np.exp(np.where(see, scale * (Q @ K.T), 0.0) - L), 0.0)
            dS = P * (D @ V.T - (D * O).sum(-1)[:, None])
            A, Gr = scale * (np.abs(Q) @ np.abs(K).T), np.abs(D) @ np.abs(V).T
            own = (np.abs(D) * np.abs(O)).sum(-1)[:, None]
            ep = (d + 8) * u * A + np.where(np.isinf(L), 0.0, 4 * u * np.abs(L)) + 16 * u
            err = (h / 3 ** 0.5 + ep) * np.abs(dS) + (d + 4) * u * P * Gr
            n = see.sum(1)[:, None]
            tiny = lambda y, axis: 2.0 ** -37 * np.abs(y).max(axis, keepdims=True) if h > 2.0 ** -24 else 0.0  # noqa: E731
            want[0][q0:q1, x] += scale * (dS @ K)
            square[0][q0:q1, x] += scale ** 2 * ((err ** 2 + see * tiny(dS, 1) ** 2 + n * (u * dS) ** 2) @ K ** 2)
            plain[0][q0:q1, x] += scale * (d + 2) * u * own * (P @ np.abs(K))
            want[1][k0:k1, e] += scale * (dS.T @ Q)
            square[1][k0:k1, e] += scale ** 2 * ((err ** 2 + see * tiny(dS, 0) ** 2).T @ Q ** 2)
            plain[1][k0:k1, e] += scale * (d + 2) * u * ((P * own).T @ np.abs(Q))
            perr = (h / 3 ** 0.5 + ep) * P
            want[2][k0:k1, e] += P.T @ D
            square[2][k0:k1, e] += (perr ** 2 + see * tiny(P, 0) ** 2).T @ D ** 2
            terms[k0:k1, e] += see.sum(0)[:, None]
    out = []
    for i, (w, sq, pl, like) in enumerate(zip(want, square, plain, (q, k, v))):
        room = 6 * np.sqrt(sq) + pl
        if i:                                                    # the sum over queries, in fp32
            room = room + 6 * np.sqrt(terms) * u * np.abs(w)
        out.append((w.reshape(like.shape), (room + 4 * u * np.abs(w)).reshape(like.shape)))    # scale, at the store
    return out
