"""Windowed attention with sinks against the fp64 oracle, element by element.

Bounds.  u = 2^-24, h = half a step of the type (2^-8, 2^-11, or 2^-24).  A score is a sum
of d products in fp32 in some order: off by at most (d + 2) u A, A = scale max_j sum |q| |k_j|; with the
exponential's own error (2 units in the last place of exp2, and its argument's rounding, 2 u (|s| + |max|) log2 e) a
probability is off by e_p = (d + 8) u A + 16 u relative, A >= |s|.  As an operand it is rounded to the type: h.  The sum
of n of them adds (n + 8) u.  So with B = max|v| over what is seen,
  |o - o'| <= 2 (e_p + (n + 8) u + h) * B   (weights sum to one; the sum's own error once more),
and o is rounded once: within() adds that.  lse: e_p + (n + 8) u + 8 u |lse|.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn
from oracle import attention as A

from .op_util import HALF, U, cu_tensor, dev, host, within

pytestmark = pytest.mark.gpu


def inputs(seed, B, T, Tk, H, KV, d, dtype, spread=1.0):
    g = np.random.default_rng(seed)
    t = [dev(spread * g.standard_normal((B, n, h, d)), dtype) for n, h in ((T, H), (Tk, KV), (Tk, KV))]
    return t, [host(x) for x in t]


def errors(q, k, scale):
    """e_p of the header, from the largest scores of the call."""
    d = q.shape[-1]
    a = scale * np.abs(q).max() * np.abs(k).sum(-1).max() if k.size and q.size else 0.0
    return (d + 8) * U * a + 16 * U


def check(t, x, dtype, window, sinks, cu=None, cuk=None, scale=None, label=""):
    q, k, v = x
    s = q.shape[-1] ** -0.5 if scale is None else scale
    o, lse = gdn.swa_fwd(*t, window, sinks, cu_tensor(cu), cu_tensor(cuk), scale=scale)
    torch.cuda.synchronize()
    ro, rl = A.attention(q, k, v, window, sinks, cu, cuk, scale)
    n = min(k.shape[1], window + sinks)
    e = errors(q, k, s) + (n + 8) * U
    big = np.abs(v).max() if v.size else 0.0
    within(o, ro, 2 * (e + HALF[dtype]) * big, dtype, f"{label} o")
    gone = rl == -np.inf
    assert np.array_equal(host(lse) == -np.inf, gone)
    assert not host(o)[gone].any()
    within(torch.where(torch.isinf(lse), 0.0, lse), np.where(gone, 0.0, rl),
           e + 8 * U * np.abs(np.where(gone, 0.0, rl)).max(initial=0.0), "fp32", f"{label} lse")
    return o, lse, ro, rl


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("T,H,KV,window,sinks", [
    (1, 1, 1, 1, 0), (2, 4, 2, 1, 1), (31, 3, 3, 5, 0), (33, 2, 1, 7, 2), (64, 2, 2, 64, 0), (65, 6, 2, 1000, 3),
    (200, 4, 4, 33, 1), (257, 2, 1, 100, 40), (130, 16, 1, 50, 4)])
def test_shapes(dtype, d, T, H, KV, window, sinks):
    if dtype == "fp32" and d == 256:
        pytest.skip("fp32 is built to 128")
    t, x = inputs(d + T, 2, T, T, H, KV, d, dtype)
    check(t, x, dtype, window, sinks, label=f"{dtype} d{d} T{T} H{H}/{KV} W{window} S{sinks}")


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 12, 16])
def test_groups(group):
    """Heads per key head that do and do not divide a tile's rows."""
    t, x = inputs(group, 1, 150, 150, 2 * group, 2, 64, "bf16")
    check(t, x, "bf16", 40, 2, label=f"group {group}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed(dtype):
    cu = [0, 0, 1, 66, 66, 67, 300, 300]
    t, x = inputs(5, 1, 300, 300, 4, 2, 64, dtype)
    check(t, x, dtype, 70, 2, cu, label="packed")
    check(t, x, dtype, 1 << 30, 0, cu, label="packed causal")


@pytest.mark.parametrize("T", [1, 40, 150])
def test_more_keys_than_queries(T):
    t, x = inputs(T, 2, T, 500, 4, 2, 64, "bf16")
    check(t, x, "bf16", 100, 3, label="behind 500 keys")
    cu, cuk = [0, T, T, 2 * T], [0, 300, 400, 1000]
    t, x = inputs(T + 1, 1, 2 * T, 1000, 4, 2, 64, "bf16")
    check(t, x, "bf16", 128, 4, cu, cuk, label="packed behind keys")


def test_rows_that_see_nothing():
    """More queries than keys: the first stand before every key."""
    t, x = inputs(9, 2, 100, 30, 4, 2, 32, "fp16")
    check(t, x, "fp16", 16, 2, label="fewer keys")
    cu, cuk = [0, 50, 100], [0, 0, 30]
    t, x = inputs(10, 1, 100, 30, 4, 2, 32, "fp16")
    o, lse, _, _ = check(t, x, "fp16", 16, 2, cu, cuk, label="a sequence without keys")
    assert not o[0, :50].any() and (lse[0, :50] == -float("inf")).all()


def test_no_tokens():
    for T, Tk in ((0, 0), (0, 7)):
        o, lse = gdn.swa_fwd(*(torch.empty(2, n, 2, 32, device="cuda") for n in (T, Tk, Tk)), 4)
        assert o.shape == (2, 0, 2, 32) and lse.shape == (2, 0, 2)
    q, k = torch.randn(2, 5, 2, 32, device="cuda"), torch.empty(2, 0, 2, 32, device="cuda")
    o, lse = gdn.swa_fwd(q, k, k, 4)
    assert not o.any() and (lse == -float("inf")).all()


@pytest.mark.parametrize("scale", [1e-3, 3.0])
def test_scales_and_wide_scores(scale):
    """Scores from near 0 to several hundred, growing along the keys, so that the maximum moves."""
    t, x = inputs(3, 1, 300, 300, 2, 1, 64, "fp32")
    t[1] *= torch.linspace(0.1, 4, 300, device="cuda")[None, :, None, None]
    x[1] = host(t[1])
    check(t, x, "fp32", 200, 5, scale=scale, label=f"scale {scale}")


def test_long_window_long_sequence():
    """Many tiles of keys a row, on a sample of rows."""
    t, x = inputs(12, 1, 5000, 5000, 2, 1, 128, "bf16")
    o, lse = gdn.swa_fwd(*t, 4000, 128)
    for i in (0, 127, 128, 129, 3999, 4127, 4128, 4999):
        ro, rl = A.attention(x[0][:, i:i + 1], x[1][:, :i + 1], x[2][:, :i + 1], 4000, 128)
        e = errors(*x[:2], 128 ** -0.5) + 5008 * U
        within(o[:, i:i + 1], ro, 2 * (e + HALF["bf16"]) * np.abs(x[2]).max(), "bf16", f"row {i}")
        within(lse[:, i:i + 1], rl, e + 80 * U, "fp32", f"lse {i}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_hidden_values_do_not_count(dtype, bad):
    """Keys and values that a query does not see may be anything: later tokens, tokens behind the window, the
    other sequences of a packed batch.  Where they are seen they count as a softmax counts them."""
    cu, window, sinks = [0, 90, 200], 20, 2
    t, x = inputs(21, 1, 200, 200, 4, 2, 64, dtype)
    clean, clean_lse = gdn.swa_fwd(*t, window, sinks, cu_tensor(cu))
    for where in (40, 89, 90, 150):
        q, k, v = (y.clone() for y in t)
        v[0, where, 1, 7] = bad
        o, lse = gdn.swa_fwd(q, k, v, window, sinks, cu_tensor(cu))
        first, last = (0, 90) if where < 90 else (90, 200)
        sees = torch.zeros(200, dtype=torch.bool, device="cuda")
        sees[where:min(where + window, last)] = True
        if where - first < sinks:
            sees[where:last] = True
        touched = torch.zeros_like(o, dtype=torch.bool)
        touched[0, sees, 2:, 7] = True
        assert torch.equal(o[~touched], clean[~touched]) and torch.equal(lse, clean_lse), where
        got = o[touched]
        assert torch.isnan(got).all() if np.isnan(bad) else (got == bad).all(), where
        q, k, v = (y.clone() for y in t)
        k[0, where, 0, 3] = float("nan")
        o, lse = gdn.swa_fwd(q, k, v, window, sinks, cu_tensor(cu))
        touched = torch.zeros_like(lse, dtype=torch.bool)
        touched[0, sees, :2] = True
        assert torch.equal(o[~touched], clean[~touched]) and torch.equal(lse[~touched], clean_lse[~touched]), where
        assert torch.isnan(o[touched]).all() and torch.isnan(lse[touched]).all(), where


@pytest.mark.parametrize("cu,cuk,code", [
    ([1, 50, 100], [0, 50, 100], 1), ([0, 60, 50, 100], [0, 50, 60, 100], 2), ([0, 50, 99], [0, 50, 100], 3),
    ([0, 50, 100], [-1, 50, 100], 4), ([0, 50, 60, 100], [0, 60, 50, 100], 5), ([0, 50, 100], [0, 50, 101], 6)])
def test_malformed_offsets_write_nothing(cu, cuk, code):
    t, _ = inputs(4, 1, 100, 100, 2, 1, 32, "bf16")
    o = torch.full((1, 100, 2, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    gdn.swa_fwd(*t, 10, 1, cu_tensor(cu), cu_tensor(cuk), o=o, workspace=ws)
    assert gdn.chunk_fwd_check(ws) == code and (o == 7).all()


def test_many_sequences():
    """More sequences than the table kernel has threads, empty ones among them."""
    g = np.random.default_rng(8)
    lens = g.integers(0, 4, 2500)
    cu = [0] + np.cumsum(lens).tolist()
    t, x = inputs(8, 1, cu[-1], cu[-1], 2, 1, 32, "fp32")
    check(t, x, "fp32", 2, 1, cu, label="2500 sequences")


def test_equal_calls_other_streams_and_graphs():
    t, _ = inputs(31, 1, 500, 500, 4, 2, 64, "bf16")
    cu = cu_tensor([0, 123, 500])
    o, lse = gdn.swa_fwd(*t, 100, 4, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, lse2 = gdn.swa_fwd(*t, 100, 4, cu)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = gdn.swa_fwd(*t, 100, 4, cu)
    for seed in range(3):
        for x in t:
            x.copy_(torch.randn(x.shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        o, lse = gdn.swa_fwd(*t, 100, 4, cu)
        assert torch.equal(o, o3) and torch.equal(lse, lse3)
