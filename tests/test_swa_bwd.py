"""Gradients of windowed attention with sinks against the fp64 oracle and against differences.

Bounds, u = 2^-24, h = half a step of the type.  As in the forward test a probability P is off by e_p relative (scores
of d products, the exponential), and is rounded to the type as an operand (h).  With G = max |row of d_o| (2-norm),
V = max |row of v|, X = G V >= |dP|, |D| (o is a mean of rows of v): dP and D are each off by (d + 2) u X, so
  dS = P (dP - D) is off by P (2 (d + 2) u X + 2 X e_p), and as an operand by h P 2 X more.
A row's P add to one, so
  |dq - dq'| <= scale 2 X (e_p + (d + n + 10) u + h) max|k|   (n terms of the sum: n u),
and with C = the largest sum over queries of P of one key (from the oracle's own P, at most rows seen)
  |dk - dk'| <= the same with max|q| C,   |dv - dv'| <= 2 (e_p + (n + 10) u + h) C max|d_o|.
The results are rounded once: within() adds that.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn
from oracle import attention as A

from .op_util import HALF, U, cu_tensor, dev, host, within
from .test_swa import errors, inputs

pytestmark = pytest.mark.gpu


def column_sums(q, k, lse, window, sinks, cu, cuk, scale):
    """C of the header: the largest sum of probabilities that one key gets."""
    ones = np.ones(q.shape)
    zero = np.zeros(k.shape)
    return A.attention_bwd(ones, q, k, zero, np.zeros(q.shape), lse, window, sinks, cu, cuk, scale)[2].max(initial=0.0)


def check(t, x, dtype, window, sinks, cu=None, cuk=None, scale=None, seed=0, label=""):
    q, k, v = x
    d = q.shape[-1]
    s = d ** -0.5 if scale is None else scale
    c, ck = cu_tensor(cu), cu_tensor(cuk)
    o, lse = gdn.swa_fwd(*t, window, sinks, c, ck, scale=scale)
    g = dev(np.random.default_rng(seed).standard_normal(q.shape), dtype)
    got = gdn.swa_bwd(g, *t, o, lse, window, sinks, c, ck, scale=scale)
    torch.cuda.synchronize()
    do, ho, hl = host(g), host(o), host(lse)
    want = A.attention_bwd(do, q, k, v, ho, hl, window, sinks, cu, cuk, scale)
    e = errors(q, k, s)
    n = q.shape[0] * q.shape[1] * (q.shape[2] // k.shape[2]) + min(k.shape[1], window + sinks)
    norm = lambda y: np.sqrt((y ** 2).sum(-1)).max(initial=0.0)     # noqa: E731
    X = norm(do) * norm(v)
    C = column_sums(q, k, hl, window, sinks, cu, cuk, s)
    ds = s * 2 * X * (e + (d + n + 10) * U + HALF[dtype])
    within(got[0], want[0], ds * np.abs(k).max(initial=0.0), dtype, f"{label} dq")
    within(got[1], want[1], ds * np.abs(q).max(initial=0.0) * C, dtype, f"{label} dk")
    within(got[2], want[2], 2 * (e + (n + 10) * U + HALF[dtype]) * C * np.abs(do).max(initial=0.0), dtype, f"{label} dv")
    return (g, *t, o, lse), got


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("T,H,KV,window,sinks", [
    (1, 1, 1, 1, 0), (2, 4, 2, 1, 1), (31, 3, 3, 5, 0), (33, 2, 1, 7, 2), (64, 2, 2, 64, 0), (130, 6, 2, 1000, 3),
    (200, 2, 2, 33, 1), (257, 2, 1, 100, 40)])
def test_shapes(dtype, d, T, H, KV, window, sinks):
    t, x = inputs(d + T, 2, T, T, H, KV, d, dtype)
    check(t, x, dtype, window, sinks, label=f"{dtype} d{d} T{T} H{H}/{KV} W{window} S{sinks}")


@pytest.mark.parametrize("group", [1, 3, 4, 5, 7, 8, 12, 16])
def test_groups(group):
    t, x = inputs(group, 1, 100, 100, 2 * group, 2, 64, "bf16")
    check(t, x, "bf16", 40, 2, label=f"group {group}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed(dtype):
    cu = [0, 0, 1, 66, 66, 67, 300, 300]
    t, x = inputs(5, 1, 300, 300, 4, 2, 64, dtype)
    check(t, x, dtype, 70, 2, cu, label="packed")
    check(t, x, dtype, 1 << 30, 0, cu, label="packed causal")


@pytest.mark.parametrize("dtype,sinks,group", [("bf16", 1, 2), ("fp32", 4, 1), ("fp16", 33, 3), ("bf16", 128, 1)])
def test_far_parts_of_the_sinks(dtype, sinks, group):
    """Tokens past the window of the first keys: several parts, in batches and packed sequences of which some have
    none, with keys in front of the queries as well."""
    t, x = inputs(sinks, 1, 2300, 2300, group, 1, 32, dtype)
    check(t, x, dtype, 20, sinks, label=f"far parts, {sinks} sinks")
    cu = [0, 1300, 1300, 1340, 2300]
    check(t, x, dtype, 20, sinks, cu, label=f"far parts packed, {sinks} sinks")
    t, x = inputs(sinks, 1, 1200, 1500, group, 1, 32, dtype)
    check(t, x, dtype, 20, sinks, label="behind keys")
    check(t, x, dtype, 20, sinks, [0, 100, 1200], [0, 250, 1500], label="packed behind keys")


def test_rows_that_see_nothing():
    t, x = inputs(9, 2, 100, 30, 4, 2, 32, "fp16")
    check(t, x, "fp16", 16, 2, label="fewer keys")
    t, x = inputs(10, 1, 100, 30, 4, 2, 32, "fp32")
    _, got = check(t, x, "fp32", 16, 2, [0, 50, 100], [0, 0, 30], label="a sequence without keys")
    assert not got[0][0, :50].any()


def test_no_tokens():
    q, k = torch.empty(2, 0, 2, 32, device="cuda"), torch.randn(2, 7, 2, 32, device="cuda")
    dq, dk, dv = gdn.swa_bwd(q, q, k, k, q, torch.empty(2, 0, 2, device="cuda"), 4, 1)
    assert dq.shape == q.shape and not dk.any() and not dv.any()
    q, k = torch.randn(2, 5, 2, 32, device="cuda"), torch.empty(2, 0, 2, 32, device="cuda")
    o, lse = gdn.swa_fwd(q, k, k, 4)
    dq, dk, dv = gdn.swa_bwd(q, q, k, k, o, lse, 4)
    assert not dq.any() and dk.shape == k.shape


def test_against_differences():
    """Central differences, in 64 bits, of the loss of the oracle's forward pass."""
    window, sinks, scale = 4, 1, 0.4
    t, x = inputs(2, 1, 9, 9, 2, 1, 32, "fp32")
    w = np.random.default_rng(3).standard_normal((1, 9, 2, 32))
    o, lse = gdn.swa_fwd(*t, window, sinks, scale=scale)
    got = [host(y) for y in gdn.swa_bwd(dev(w), *t, o, lse, window, sinks, scale=scale)]
    w = host(dev(w))
    for which in range(3):
        flat = x[which].reshape(-1)
        for at in range(0, flat.size, 7):
            keep, side = flat[at], []
            for step in (1e-5, -1e-5):
                flat[at] = keep + step
                side.append((A.attention(*x, window, sinks, scale=scale)[0] * w).sum())
            flat[at] = keep
            # differences: 1e-10 from the step, 1e-9 from cancellation; the kernel: fp32 over some 32 products
            assert abs(got[which].reshape(-1)[at] - (side[0] - side[1]) / 2e-5) <= 1e-5 * max(1, np.abs(got[which]).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_hidden_values_do_not_count(dtype, bad):
    """A value that is not finite reaches the gradients of what sees it, or is seen by it, alone."""
    cu, window, sinks = [0, 90, 200], 20, 2
    t, x = inputs(21, 1, 200, 200, 4, 2, 64, dtype)
    c = cu_tensor(cu)
    o, lse = gdn.swa_fwd(*t, window, sinks, c)
    g = dev(np.random.default_rng(5).standard_normal(t[0].shape), dtype)
    clean = gdn.swa_bwd(g, *t, o, lse, window, sinks, c)
    for where in (40, 89, 90, 150):
        first, last = (0, 90) if where < 90 else (90, 200)
        j = torch.arange(200, device="cuda")
        own = (j >= first) & (j < last)
        seen_by = own & (j >= where) & ((j - where < window) | (where - first < sinks))     # queries that see key `where`
        sees = own & (j <= where) & ((where - j < window) | (j - first < sinks))            # keys that query `where` sees
        shares = torch.zeros_like(own)                     # keys that some query of seen_by sees
        for i in torch.nonzero(seen_by)[:, 0].tolist():
            shares |= own & (j <= i) & ((i - j < window) | (j - first < sinks))
        for what in ("key", "query", "gradient"):
            q, k, v, gg = (y.clone() for y in (*t, g))
            {"key": k, "query": q, "gradient": gg}[what][0, where, 1 if what == "key" else 2, 3] = bad
            dq, dk, dv = gdn.swa_bwd(gg, q, k, v, o, lse, window, sinks, c)
            rows, cols = torch.zeros_like(dq, dtype=torch.bool), torch.zeros_like(dk, dtype=torch.bool)
            if what == "key":
                rows[0, seen_by, 2:] = True
                cols[0, shares, 1] = True
            else:
                rows[0, where, 2] = True
                cols[0, sees, 1] = True
            assert torch.equal(dq[~rows], clean[0][~rows]), (what, where)
            assert torch.equal(dk[~cols], clean[1][~cols]) and torch.equal(dv[~cols], clean[2][~cols]), (what, where)
            assert not torch.isfinite(dq[rows]).all()


def test_malformed_offsets_write_nothing():
    t, _ = inputs(4, 1, 100, 100, 2, 1, 32, "bf16")
    o, lse = gdn.swa_fwd(*t, 10, 1)
    for cu, cuk, code in (([0, 60, 50, 100], [0, 50, 60, 100], 2), ([0, 50, 100], [0, 50, 101], 6)):
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        gdn.swa_bwd(o, *t, o, lse, 10, 1, cu_tensor(cu), cu_tensor(cuk), workspace=ws)
        assert gdn.chunk_fwd_check(ws) == code


def test_equal_calls_other_streams_and_graphs():
    t, _ = inputs(31, 1, 1500, 1500, 4, 2, 64, "bf16")
    c = cu_tensor([0, 123, 1500])
    g = torch.randn_like(t[0])
    o, lse = gdn.swa_fwd(*t, 50, 4, c)
    want = gdn.swa_bwd(g, *t, o, lse, 50, 4, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = gdn.swa_bwd(g, *t, o, lse, 50, 4, c)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, lse2 = gdn.swa_fwd(*t, 50, 4, c)
        got = gdn.swa_bwd(g, *t, o2, lse2, 50, 4, c)
    for seed in range(3):
        for y in (*t, g):
            y.copy_(torch.randn(y.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        o, lse = gdn.swa_fwd(*t, 50, 4, c)
        want = gdn.swa_bwd(g, *t, o, lse, 50, 4, c)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 128), ("fp32", 64)])
def test_graphs_of_the_wide_kernels(dtype, d):
    """Kernels with more than 64 KiB of LDS, and those whose key side is split, captured and replayed."""
    t, _ = inputs(32, 2, 300, 300, 4, 2, d, dtype)
    g = torch.randn_like(t[0])
    graph = torch.cuda.CUDAGraph()
    o, lse = gdn.swa_fwd(*t, 40, 3)
    gdn.swa_bwd(g, *t, o, lse, 40, 3)
    with torch.cuda.graph(graph):
        o, lse = gdn.swa_fwd(*t, 40, 3)
        got = gdn.swa_bwd(g, *t, o, lse, 40, 3)
    for seed in range(3):
        for y in (*t, g):
            y.copy_(torch.randn(y.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        o2, lse2 = gdn.swa_fwd(*t, 40, 3)
        want = gdn.swa_bwd(g, *t, o2, lse2, 40, 3)
        assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_keys_that_repeat_the_queries_tensor():
    """One tensor as q, k and v, as the gradients of a shared projection need it."""
    t, x = inputs(40, 1, 70, 70, 2, 2, 32, "fp32")
    check([t[0]] * 3, [x[0]] * 3, "fp32", 16, 1, label="q = k = v")
