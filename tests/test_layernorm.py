"""Layer norm and its gradient on the GPU against the fp64 oracle.

Bounds.  A sum of n fp32 terms taken in any order is off by at most
(longest chain of additions) u sum|terms|; here a thread adds at most
n / 8 terms before lanes and waves join (12 more), so n / 8 + 16 covers every
layout for n <= 16384.  The worst case is used throughout.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn
from oracle import operators as R

from .op_util import DT, U, dev, host, within

pytestmark = pytest.mark.gpu

TYPES = [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "bf16"), ("bf16", "fp32"), ("fp32", "fp16"),
         ("fp16", "fp32")]
DIMS = [1, 2, 7, 8, 16, 24, 63, 64, 65, 100, 128, 136, 255, 256, 264, 512, 513, 768, 1000, 1001, 1024, 1032, 2048,
        2049, 4096, 4104, 5000, 8192, 8200, 8201, 12000, 16376, 16383, 16384]


def chain(n):
    return (n / 8 + 16) * U


def stats_bound(x, D, eps):
    """Errors of the mean and, relative, of rstd."""
    dm = chain(D) * np.abs(x).mean(1) + U * np.abs(x.mean(1))
    c = x - x.mean(1, keepdims=True)
    var = (c * c).mean(1)
    # c_i is off by dm + u |c_i|: its square's sum by 2 sum|c| (dm + u|c|) + n dm^2, then the sum's own chain
    dc = dm[:, None] + U * np.abs(c)
    dv = (2 * np.abs(c) * dc + dc * dc).mean(1) + (chain(D) + 3 * U) * var
    return dm, dv / (var + eps) / 2 + 4 * U + (dv / (var + eps)) ** 2


def make(R_, D, types, seed=0, shift=0.0):
    g = np.random.default_rng(seed)
    x = dev(g.standard_normal((R_, D)) * g.uniform(0.2, 3, (R_, 1)) + shift + g.standard_normal((R_, 1)), types[0])
    return x, dev(1 + 0.3 * g.standard_normal(D)), dev(g.standard_normal(D)), dev(g.standard_normal((R_, D)), types[1])


def check_fwd(rows, D, types, seed=0, weight=True, bias=True, shift=0.0, eps=1e-5):
    x, w, b, _ = make(rows, D, types, seed, shift)
    w, b = w if weight else None, b if bias else None
    y, mean, rstd = gdn.layernorm_fwd(x, w, b, eps=eps, out_dtype=DT[types[1]])
    xr = host(x)
    want, wm, wr = R.layernorm(xr, None if w is None else host(w), None if b is None else host(b), eps)
    dm, dr = stats_bound(xr, D, eps)
    within(mean, wm, dm, "fp32", f"mean {rows, D} {types}")
    within(rstd, wr, dr * wr, "fp32", "rstd")
    aw = 1.0 if w is None else np.abs(host(w))
    c = np.abs(xr - wm[:, None])
    room = wr[:, None] * ((dm[:, None] + 2 * U * c) * (1 + dr[:, None]) + c * (dr[:, None] + 3 * U)) * aw
    # y may also be formed as x (rstd w) + (b - mean rstd w)
    room += 3 * U * (np.abs(want) + (0 if b is None else np.abs(host(b))))
    within(y, want, room, types[1], "y")
    return x, w, b, y, mean, rstd


def check_bwd(rows, D, types, seed=0, weight=True, shift=0.0):
    x, w, _, dy = make(rows, D, types, seed, shift)
    w = w if weight else None
    _, wm, wr = R.layernorm(host(x))
    mean, rstd = dev(wm), dev(wr)
    got = gdn.layernorm_bwd(dy, x, mean, rstd, w)
    m, r, xr, dyr = host(mean), host(rstd), host(x), host(dy)
    wx, ww, wb = R.layernorm_bwd(dyr, xr, m, r, None if w is None else host(w))
    xh = np.abs((xr - m[:, None]) * r[:, None])
    u = np.abs(dyr if w is None else dyr * host(w))
    e1 = (chain(D) + 2 * U) * u.mean(1, keepdims=True)
    e2 = (chain(D) + 6 * U) * (u * xh).mean(1, keepdims=True)
    room = r[:, None] * (5 * U * u + e1 + xh * e2
                         + 6 * U * (u.mean(1, keepdims=True) + xh * (u * xh).mean(1, keepdims=True)))
    within(got[0], wx, room, types[0], f"dx {rows, D} {types}")
    # a column's chain: the rows that one thread adds, then at most 64 joins twice over
    rc = (rows / 4 + 140) * U
    within(got[1], ww, rc * (np.abs(dyr) * xh).sum(0), "fp32", "dweight")
    within(got[2], wb, rc * np.abs(dyr).sum(0), "fp32", "dbias")
    return x, w, dy, mean, rstd, got


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("D", [128, 100, 1001, 2048])
def test_types(D, types):
    check_fwd(37, D, types)
    check_bwd(37, D, types)


@pytest.mark.parametrize("D", DIMS)
def test_dims(D):
    for types in (("bf16", "bf16"), ("fp32", "fp32")):
        check_fwd(5, D, types, seed=D)
        check_bwd(5, D, types, seed=D)


@pytest.mark.parametrize("rows", [1, 2, 3, 31, 64, 1000, 4097])
def test_rows(rows):
    for D in (128, 33, 520):
        check_fwd(rows, D, ("bf16", "bf16"), seed=rows)
        check_bwd(rows, D, ("bf16", "fp32"), seed=rows)


def test_without_parameters_and_stats():
    for kw in (dict(weight=False), dict(bias=False), dict(weight=False, bias=False)):
        x, w, b, y, _, _ = check_fwd(9, 72, ("bf16", "bf16"), **kw)
        y2, m, r = gdn.layernorm_fwd(x, w, b, out_dtype=torch.bfloat16, stats=False)
        assert m is None and r is None and torch.equal(y, y2)
    x, w, dy, mean, rstd, got = check_bwd(9, 72, ("bf16", "bf16"), weight=False)
    ones = gdn.layernorm_bwd(dy, x, mean, rstd, torch.ones(72, device="cuda"))
    assert all(torch.equal(p, q) for p, q in zip(got, ones))
    for dw in (True, False):
        for db in (True, False):
            part = gdn.layernorm_bwd(dy, x, mean, rstd, w, dweight=dw, dbias=db)
            assert torch.equal(part[0], got[0])
            assert torch.equal(part[1], got[1]) if dw else part[1] is None
            assert torch.equal(part[2], got[2]) if db else part[2] is None


def test_far_mean_and_constant_rows():
    """The variance is taken about the mean: rows far from zero keep theirs, constant rows give the bias."""
    check_fwd(16, 256, ("fp32", "fp32"), shift=1000.0)
    check_fwd(16, 250, ("fp32", "fp32"), shift=-300.0)
    for D in (64, 100, 2048):     # sums of an exact constant are exact: the mean is the constant
        x = torch.full((3, D), 0.5, device="cuda")
        b = torch.randn(D, device="cuda")
        y, mean, rstd = gdn.layernorm_fwd(x, torch.randn(D, device="cuda"), b, eps=1e-5)
        assert torch.equal(y, b.expand(3, D)) and (mean == 0.5).all()
        assert torch.allclose(rstd, torch.full_like(rstd, 1e-5).rsqrt(), rtol=1e-6, atol=0)


def test_bad_row_stays_alone():
    x, w, b, dy = make(50, 136, ("fp32", "fp32"))
    y, mean, rstd = gdn.layernorm_fwd(x, w, b)
    dx = gdn.layernorm_bwd(dy, x, mean, rstd, w)[0]
    bad = x.clone()
    bad[17, 5] = float("nan")
    bad[18] = float("inf")
    y2, m2, r2 = gdn.layernorm_fwd(bad, w, b)
    keep = [i for i in range(50) if i not in (17, 18)]
    assert torch.equal(y[keep], y2[keep]) and y2[17:19].isnan().all()
    dx2 = gdn.layernorm_bwd(dy, bad, m2, r2, w)[0]
    assert torch.equal(dx[keep], dx2[keep])


def test_empty():
    x = torch.empty(0, 24, device="cuda")
    y, mean, rstd = gdn.layernorm_fwd(x)
    assert y.shape == (0, 24) and mean.shape == (0,)
    dx, dw, db = gdn.layernorm_bwd(y, x, mean, rstd)
    assert dx.shape == (0, 24) and not dw.any() and not db.any() and dw.shape == (24,)


def test_leading_dims():
    x = torch.randn(2, 3, 5, 40, device="cuda", dtype=torch.bfloat16)
    y, mean, rstd = gdn.layernorm_fwd(x)
    assert y.shape == x.shape and mean.shape == (2, 3, 5)
    flat = gdn.layernorm_fwd(x.view(30, 40))
    assert torch.equal(y.view(30, 40), flat[0]) and torch.equal(mean.view(30), flat[1])
    dx, dw, db = gdn.layernorm_bwd(y, x, mean, rstd)
    assert dx.shape == x.shape
    x1 = x[0, 0, 0].contiguous()
    assert torch.equal(gdn.layernorm_fwd(x1)[0], y[0, 0, 0])


def test_gradient_equals_differences():
    """dx, dw, db against central differences of the loss in fp64 (error step^2), and against the fp64 formula."""
    x, w, b, dy = make(6, 40, ("fp32", "fp32"), seed=3)
    y, mean, rstd = gdn.layernorm_fwd(x, w, b)
    got = [host(v) for v in gdn.layernorm_bwd(dy, x, mean, rstd, w)]
    v, d = [host(x), host(w), host(b)], host(dy)
    loss = lambda v: (d * R.layernorm(*v)[0]).sum()                      # noqa: E731
    g = np.random.default_rng(5)
    for i in range(3):
        way = g.standard_normal(v[i].shape)
        hi, lo = list(v), list(v)
        hi[i], lo[i] = v[i] + 1e-5 * way, v[i] - 1e-5 * way
        want, have = (loss(hi) - loss(lo)) / 2e-5, (got[i] * way).sum()
        # fp32 sums of at most 240 terms in got, and the statistics' rounding
        assert abs(want - have) <= 400 * U * (np.abs(got[i]) * np.abs(way)).sum() + 400 * U * np.abs(d).sum() + 1e-6


def test_equal_bits_streams_and_graph():
    x, w, b, dy = make(3000, 264, ("bf16", "bf16"))
    ref = gdn.layernorm_fwd(x, w, b, out_dtype=torch.bfloat16)
    gref = gdn.layernorm_bwd(dy, x, ref[1], ref[2], w)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            got.append(gdn.layernorm_fwd(x, w, b, out_dtype=torch.bfloat16) + gdn.layernorm_bwd(dy, x, *ref[1:], w))
    torch.cuda.synchronize()
    for v in got:
        assert all(torch.equal(p, q) for p, q in zip(v, ref + gref))
    y = torch.empty_like(ref[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, mean, rstd = gdn.layernorm_fwd(x, w, b, y=y)
        grads = gdn.layernorm_bwd(dy, x, mean, rstd, w)
    for k in range(4):
        x.normal_()
        dy.normal_()
        graph.replay()
        torch.cuda.synchronize()
        e = gdn.layernorm_fwd(x, w, b, out_dtype=torch.bfloat16)
        eg = gdn.layernorm_bwd(dy, x, *e[1:], w)
        assert all(torch.equal(p, q) for p, q in zip((y, mean, rstd) + grads, e + eg))


def test_offsets_past_32_bits():
    rows, D = 2_200_000, 1000
    x = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.rand(D, device="cuda")
    y, mean, rstd = gdn.layernorm_fwd(x, w, out_dtype=torch.bfloat16)
    part = gdn.layernorm_fwd(x[-9:].clone(), w, out_dtype=torch.bfloat16)
    assert torch.equal(y[-9:], part[0]) and torch.equal(mean[-9:], part[1]) and torch.equal(rstd[-9:], part[2])
    dx, dw, db = gdn.layernorm_bwd(y, x, mean, rstd, w)
    assert torch.equal(dx[-9:], gdn.layernorm_bwd(y[-9:].clone(), x[-9:].clone(), *part[1:], w)[0])
    # worst case of test bounds on columns of 2.2 million rows would say nothing: a random walk's size does
    want = y.sum(0, dtype=torch.float64)
    assert ((db.double() - want).abs() <= 1e-4 * y.float().abs().sum(0, dtype=torch.float64)).all()


def test_refusals():
    x = torch.randn(6, 10, device="cuda")
    for bad in (x.t(), x[:, ::2]):
        with pytest.raises(ValueError, match="contiguous"):
            gdn.layernorm_fwd(bad)
    with pytest.raises(ValueError, match="dtype"):
        gdn.layernorm_fwd(x.double())
    with pytest.raises(ValueError, match="dtype"):
        gdn.layernorm_fwd(x, torch.ones(10, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="must be"):
        gdn.layernorm_fwd(x, torch.ones(9, device="cuda"))
    with pytest.raises(gdn.GdnError, match="mix"):
        gdn.layernorm_fwd(x.bfloat16(), out_dtype=torch.float16)
    with pytest.raises(gdn.GdnError, match="eps"):
        gdn.layernorm_fwd(x, eps=-1.0)
    with pytest.raises(gdn.GdnError, match="aligned"):
        gdn.layernorm_fwd(x.view(-1)[1:11].view(1, 10))
    with pytest.raises(gdn.GdnError, match="overlaps"):
        gdn.layernorm_fwd(x, y=x)
    with pytest.raises(gdn.GdnError, match="dim"):
        gdn.layernorm_fwd(torch.zeros(1, 16385, device="cuda"))
    with pytest.raises(ValueError, match="must be"):
        gdn.layernorm_bwd(x, x, x[:5, 0].contiguous(), x[:, 0].contiguous())
