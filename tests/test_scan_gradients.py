"""Gradients of the gated linear recurrence against differences of the loss, taken in 64 bits."""
import numpy as np
import pytest

import gated_delta_rule_24_amd as gdn
from oracle import operators as R

from .op_util import U, cu_tensor, host
from .test_scan import bound_scan, inputs

pytestmark = pytest.mark.gpu


def room_and_derivatives(r, h, cu):
    """Bounds of the gradients of one call: those of test_scan, and half a step of fp32 for the results."""
    B, T, D = r["x"].shape
    E, last = bound_scan(r["dh"], r["la"], r["dfin"], B, T, D, cu, reverse=True)
    wx, wl, wi = R.scan_bwd(r["la"], h, r["dh"], r["init"], r["dfin"], cu)
    past = np.zeros((B * T, D))
    for n, (t0, t1) in enumerate(R._spans(B, T, cu)):
        if t1 > t0:
            past[t0], past[t0 + 1:t1] = r["init"][n], h.reshape(-1, D)[t0:t1 - 1]
    past = np.abs(past).reshape(B, T, D)
    # h itself was rounded to fp32 on the way: a step of it in dlog_alpha
    dl = past * np.exp(r["la"]) * (E + (12 + 4 * np.abs(r["la"])) * U * np.abs(wx))
    return {"x": E + U * np.abs(wx), "la": dl + U * np.abs(wl), "init": last + U * np.abs(wi)}


@pytest.mark.parametrize("B,T,D,cu", [(1, 40, 8, [0, 10, 10, 40]), (3, 30, 5, None), (2, 200, 36, None),
                                      (1, 300, 20, [0, 1, 130, 300])])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_gradients_equal_differences(B, T, D, cu, seed):
    """The derivative along a random direction of the loss sum(h dh) + sum(final dfinal).  Central differences over
    +-s leave s^2 / 6 of the third derivative.  Along log_alpha that is taken from the differences themselves, as the
    distance of the differences at s and 2 s, which is three times what s leaves; x and init are linear.  In 64 bits
    at s = 2^-10 rounding adds 2^-52 of the loss over s.  What remains is the kernel's own bound, so that a term that
    is missing or wrong by a thousandth shows."""
    t, r = inputs(B, T, D, cu, ("fp32",) * 3, seed=10 + seed)
    cuts = cu_tensor(cu)
    h, _ = gdn.scan_fwd(t["x"], t["la"], t["init"], cuts)
    grads = dict(zip(("x", "la", "init"), gdn.scan_bwd(t["la"], h, t["dh"], t["init"], t["dfin"], cuts)))
    # h's own error reaches dlog_alpha through h_{t-1}: the bound takes the oracle's h and adds it
    exact = R.scan(r["x"], r["la"], r["init"], cu)[0]
    Eh, _ = bound_scan(r["x"], r["la"], r["init"], B, T, D, cu)
    room = room_and_derivatives(r, exact, cu)
    wx = np.abs(R.scan_bwd(r["la"], exact, r["dh"], r["init"], r["dfin"], cu)[0])
    shifted = np.concatenate([np.zeros((1, D)), Eh.reshape(-1, D)[:-1]]).reshape(B, T, D)
    room["la"] = room["la"] + shifted * np.exp(r["la"]) * wx

    def loss(v):
        h, fin = R.scan(v["x"], v["la"], v["init"], cu)
        return (h * r["dh"]).sum() + (fin * r["dfin"]).sum()

    def slope(name, way, s):
        hi, lo = dict(r), dict(r)
        hi[name], lo[name] = r[name] + s * way, r[name] - s * way
        return (loss(hi) - loss(lo)) / (2 * s)

    size = np.abs(exact * r["dh"]).sum() + np.abs(r["dfin"]).sum() * np.abs(exact).max()
    g = np.random.default_rng(seed)
    for name, got in grads.items():
        way, s = g.standard_normal(r[name].shape), 2.0 ** -10
        want, wide = slope(name, way, s), slope(name, way, 2 * s)
        have = (host(got) * way).sum()
        allowed = (room[name] * np.abs(way)).sum() + abs(wide - want) + 16 * 2.0 ** -52 * size / s
        scale = np.sqrt(((host(got) * way) ** 2).sum())
        print(f"[differences] {name}: {have:.8g} against {want:.8g}, room {allowed:.2g} of {scale:.3g}", flush=True)
        assert abs(have - want) <= allowed
        assert allowed <= 1e-2 * scale          # the comparison says something
