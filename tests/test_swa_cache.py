"""The resident cache of windowed attention and the step on it, against the fp64 oracle.

Writing moves bits or rounds once by a rule without ties to other roundings: compared bit for bit.  Reading an 8-bit
row gives value * scale rounded once: exact in bf16 and fp32, and compared after that rounding.  The step's bound is
that of the forward call (tests/test_swa.py) with the cache's own values as keys and values, which are exact.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn
from oracle import attention as A

from .op_util import DT, HALF, U, cu_tensor, dev, host, within
from .test_swa import errors

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def new_cache(seed, P, KV, rows, d, kind):
    """A cache with something in every row, as (cache, scales) on the device and as the oracle's."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((2, P, KV, rows, d))
    if kind != "e4m3":
        c = dev(x, kind)
        return c, None, host(c), None
    c = torch.from_numpy((100 * x).clip(-448, 448).astype(np.float32)).cuda().to(E4M3)
    s = torch.from_numpy(2.0 ** g.integers(-9, -3, (2, P, KV, rows)).astype(np.float32)).cuda()
    return c, s, host(c.float()), host(s)


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def same(c, s, rc, rs):
    alike = np.array_equal(host(c.float()), rc, equal_nan=True)
    assert alike, "cache"
    alike = s is None or np.array_equal(host(s), rs, equal_nan=True)
    assert alike, "scales"


@pytest.mark.parametrize("kind,dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("e4m3", "bf16"),
                                        ("e4m3", "fp16"), ("e4m3", "fp32")])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_write_and_read(kind, dtype, d):
    """Packed tokens of sequences that are new, go on, or wrap the ring several times, into slots in any order."""
    P, KV, window, sinks = 7, 3, 10, 2
    lengths, slots, cu = [0, 5, 11, 25, 3, 1], [6, 2, 0, 3, -1, 5], [0, 1, 1, 30, 41, 50, 77]
    c, s, rc, rs = new_cache(d, P, KV, window + sinks, d, kind)
    g = np.random.default_rng(d + 1)
    k, v = (dev(g.standard_normal((1, 77, KV, d)) * np.exp(3 * g.standard_normal((1, 77, KV, 1))), dtype)
            for _ in range(2))
    status = i32([9, 9])
    out = gdn.cache_write(c, k, v, i32(lengths), sinks, s, i32(slots), cu_tensor(cu), status=status)
    assert out is c and gdn.cache_check(status) == 0
    rc, rs = A.cache_write(rc, host(k), host(v), lengths, sinks, rs, slots, cu)
    same(c, s, rc, rs)

    after = [n + b - a for n, a, b in zip(lengths, cu, cu[1:])]
    k, v = gdn.cache_read(c, i32(after), sinks, s, i32(slots), out_dtype=DT[dtype])
    assert k.shape == (6, window + sinks, KV, d)
    for n, both in enumerate(A.cache_read(rc, after, sinks, rs, slots)):
        if both is None:
            continue
        for got, want in zip((k, v), both):
            # (in fp16 some inputs are infinite: those rows are NaN)
            alike = np.array_equal(host(got[n, :len(want)]), host(dev(want, dtype)), equal_nan=True)
            assert alike, n
    # packed, with room behind each sequence's rows, which keeps what it holds
    rows = [0 if b is None else len(b[0]) for b in A.cache_read(rc, after, sinks, rs, slots)]
    cuk = np.concatenate([[0], np.cumsum(np.array(rows) + 3)]).tolist()
    k2, v2 = (torch.full((1, cuk[-1], KV, d), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    gdn.cache_read(c, i32(after), sinks, s, i32(slots), cu_tensor(cuk), k=k2, v=v2, status=status)
    assert gdn.cache_check(status) == 0
    for n, (a, r) in enumerate(zip(cuk, rows)):
        bits = torch.int32 if dtype == "fp32" else torch.int16
        assert torch.equal(k2[0, a:a + r].view(bits), k[n, :r].view(bits))
        assert torch.equal(v2[0, a:a + r].view(bits), v[n, :r].view(bits))
        assert (k2[0, a + r:cuk[n + 1]] == 7).all()


@pytest.mark.parametrize("window,sinks,T,have", [(1, 0, 5, 0), (1, 1, 3, 0), (4, 3, 2, 1), (4, 3, 9, 0), (100, 128, 60, 90),
                                                 (5, 0, 5, 5), (7, 2, 1, 1 << 29)])
def test_write_rows_of_equal_length(window, sinks, T, have):
    c, s, rc, rs = new_cache(3, 2, 1, window + sinks, 32, "e4m3")
    k, v = (dev(np.random.default_rng(i).standard_normal((2, T, 1, 32)), "bf16") for i in range(2))
    gdn.cache_write(c, k, v, i32([have, have]), sinks, s)
    same(c, s, *A.cache_write(rc, host(k), host(v), [have, have], sinks, rs))


def test_e4m3_rows():
    """Every e4m3 value and the places between them, zeros, rows at the scale's borders, rows that are not finite."""
    top = torch.arange(0, 127, device="cuda", dtype=torch.uint8).view(E4M3).float()
    between = (top[1:] + top[:-1]) / 2
    near = torch.stack([torch.nextafter(between, between - 1), torch.nextafter(between, between + 1)]).reshape(-1)
    values = torch.cat([top, between, near, -top, -between, -near])
    rows = []
    for chunk in values.split(30):
        rows.append(torch.cat([chunk, chunk.new_zeros(30 - len(chunk)), chunk.new_tensor([448.0, -448.0])]))
    tiny = 2.0 ** -126
    for x in (0.0, -0.0, 448.0, 448.00003, 464.0, 1.75, 1.7500001, 3.5, 1e-40, tiny, 448 * tiny, 1e38, 3.4e38, 2.0 ** 127):
        rows.append(torch.linspace(-x, x, 32, device="cuda", dtype=torch.float64).float())
    for x in (float("nan"), float("inf"), -float("inf")):
        rows.append(torch.ones(32, device="cuda"))
        rows[-1][5] = x
    x = torch.stack(rows)[None, :, None]
    n = x.shape[1]
    c = torch.zeros(2, 1, 1, n, 32, device="cuda").to(E4M3)
    s = torch.zeros(2, 1, 1, n, device="cuda")
    gdn.cache_write(c, x.contiguous(), -x, None, 0, s)
    for side, y in ((0, x), (1, -x)):
        for r in range(n):
            want, scale = A.e4m3(host(y[0, r, 0]))
            alike = np.array_equal(host(c[side, 0, 0, r].float()), want, equal_nan=True)
            assert alike and np.array_equal(host(s[side, 0, 0, r]), scale, equal_nan=True), (side, r)
    k, _ = gdn.cache_read(c, i32([n]), 0, s, out_dtype=torch.float32)
    want = c[0, 0, 0].double() * s[0, 0, 0][:, None].double()
    assert torch.equal(torch.nan_to_num(k[0, :, 0], 7.0), torch.nan_to_num(want.float(), 7.0))


@pytest.mark.parametrize("what,lengths,slots,cu,code", [
    ("write", [0, 0], [0, 4], None, 4), ("write", [0, 0], [0, -2], None, 4), ("write", [0, 0], [1, 1], None, 5),
    ("write", [0, -1], [0, 1], None, 6), ("write", [0, (1 << 30) - 5], [0, 1], None, 6),
    ("write", [0, 0], [0, 1], [1, 5, 20], 1), ("write", [0, 0], [0, 1], [0, 21, 20], 2),
    ("write", [0, 0], [0, 1], [0, 5, 19], 3), ("read", [0, 11], [0, 1], None, 7), ("read", [3, 3], [2, 2], None, 5),
    ("read", [3, -3], [2, 1], None, 6), ("read", [3, 3], [2, 9], None, 4), ("read", [6, 6], [2, 1], [0, 5, 20], 7)])
def test_bad_indices_write_nothing(what, lengths, slots, cu, code):
    c, s, _, _ = new_cache(1, 4, 2, 12, 32, "e4m3")
    k, v = (torch.full((1, 20, 2, 32) if cu else (2, 10, 2, 32), 7.0, dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    status = i32([9, 9])
    before = c.clone(), s.clone(), k.clone()
    if what == "write":
        gdn.cache_write(c, k, v, i32(lengths), 2, s, i32(slots), cu_tensor(cu), status=status)
    else:
        gdn.cache_read(c, i32(lengths), 2, s, i32(slots), cu_tensor(cu), k=k, v=v, status=status)
    assert gdn.cache_check(status) == code
    assert torch.equal(c.view(torch.uint8), before[0].view(torch.uint8)) and torch.equal(s, before[1])
    assert torch.equal(k, before[2]) and torch.equal(v, before[2])


def test_no_sequences_and_no_tokens():
    c, s, rc, rs = new_cache(1, 4, 2, 12, 32, "e4m3")
    status = i32([9, 9])
    none = torch.empty(0, 5, 2, 32, device="cuda")
    gdn.cache_write(c, none, none, None, 2, s, status=status)
    assert status.tolist() == [0, 0]
    gdn.cache_write(c, torch.empty(3, 0, 2, 32, device="cuda"), torch.empty(3, 0, 2, 32, device="cuda"), None, 2, s)
    same(c, s, rc, rs)
    o = gdn.swa_step(c, none[:, 0], none[:, 0], none[:, 0], i32([]), 2, s, status=status.fill_(9))
    assert o.shape == (0, 2, 32) and status.tolist() == [0, 0]
    k, _ = gdn.cache_read(c, i32([0, 0]), 2, s)
    assert k.shape == (2, 12, 2, 32)


def step_check(dtype, kind, d, H, KV, window, sinks, lengths, P=None, slots=None, seed=0, scale=None):
    N = len(lengths)
    c, s, rc, rs = new_cache(seed, P or N, KV, window + sinks, d, kind)
    g = np.random.default_rng(seed + 1)
    q, k, v = (dev(g.standard_normal((N, h, d)), dtype) for h in (H, KV, KV))
    status = i32([9, 9])
    o = gdn.swa_step(c, q, k, v, i32(lengths), sinks, s, i32(slots), scale=scale, status=status)
    assert gdn.cache_check(status) == 0
    ro, rc, rs = A.step(rc, host(q), host(k), host(v), lengths, sinks, rs, slots, scale)
    same(c, s, rc, rs)
    full = rc if rs is None else rc * rs[..., None]
    n = window + sinks
    e = errors(host(q), full[0], d ** -0.5 if scale is None else scale) + (n + 8) * U
    within(o, ro, 2 * (e + HALF[dtype]) * np.abs(full[1]).max(), dtype, f"{dtype} {kind} d{d} H{H}/{KV} rows {n}")
    return o


@pytest.mark.parametrize("kind,dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("e4m3", "bf16"),
                                        ("e4m3", "fp16"), ("e4m3", "fp32")])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_step(kind, dtype, d):
    if dtype == "fp32" and d == 256:
        pytest.skip("fp32 is built to 128")
    step_check(dtype, kind, d, 6, 2, 37, 3, [0, 1, 2, 3, 36, 39, 40, 41, 200, 1 << 29], seed=d)
    step_check(dtype, kind, d, 2, 2, 300, 0, [299, 300, 7], P=5, slots=[4, 0, 2], seed=d)


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 16])
def test_step_groups(group):
    step_check("bf16", "e4m3", 64, 2 * group, 2, 70, 4, [5, 73, 74, 1000], seed=group)


@pytest.mark.parametrize("window,sinks,scale", [(1, 0, None), (1, 128, None), (1000, 4, 2.0), (5000, 128, None)])
def test_step_split_rows(window, sinks, scale):
    """One sequence: its rows split over blocks, some of which have none."""
    for length in (0, window // 2, 3 * window + 1000):
        step_check("bf16", "bf16", 64, 4, 1, window, sinks, [length], seed=window, scale=scale)
    step_check("fp16", "e4m3", 128, 4, 2, window, sinks, [window + sinks, 0, 1], P=3, slots=[2, 1, 0], seed=1)


def test_step_leaves_sequences_out():
    """Padding by slot -1; slots out of range or given twice and bad lengths, which the status tells of."""
    for lengths, slots, out, code in (([5, 9, 3], [1, -1, 0], [1], 0), ([5, 9, 3], [1, 7, 0], [1], 4),
                                      ([5, 9, 3], [1, 0, 1], [0, 2], 5), ([5, -1, 3], [0, 1, 2], [1], 6),
                                      ([5, 1 << 30, 3], [0, 1, 2], [1], 6)):
        for window in (20, 3000):
            c, s, rc, rs = new_cache(1, 4, 1, window + 2, 32, "e4m3")
            g = np.random.default_rng(2)
            q, k, v = (dev(g.standard_normal((3, h, 32)), "bf16") for h in (2, 1, 1))
            status = i32([9, 9])
            o = gdn.swa_step(c, q, k, v, i32(lengths), 2, s, i32(slots), status=status)
            assert gdn.cache_check(status) == code
            ro, rc, rs = A.step(rc, host(q), host(k), host(v), [0 if n in out else x for n, x in enumerate(lengths)], 2,
                                rs, [-1 if n in out else x for n, x in enumerate(slots)])
            same(c, s, rc, rs)
            assert not o[out].any() and np.abs(host(o) - ro).max() <= 0.05


def test_step_values_not_finite():
    """Rows past the sequence's end hold anything; a row that is not finite is seen as such."""
    c, _, rc, _ = new_cache(1, 2, 1, 200, 64, "bf16")
    c[:, 0, :, 50:] = float("nan")
    q, k, v = (torch.randn(2, h, 64, device="cuda").bfloat16() for h in (2, 1, 1))
    clean = c.clone()
    clean[:, 0, :, 50:] = 0
    o = gdn.swa_step(c, q, k, v, i32([20, 150]))
    assert torch.equal(o, gdn.swa_step(clean, q, k, v, i32([20, 150]))) and torch.isfinite(o).all()
    c[1, 1, 0, 33, 4] = float("inf")
    o = gdn.swa_step(c, q, k, v, i32([20, 150]))
    assert (o[1, :, 4] == float("inf")).all() and torch.isfinite(o[0]).all()


def test_step_in_a_graph():
    """A captured step, replayed with lengths that its caller moves on, against eager calls on a copy."""
    c, s, _, _ = new_cache(5, 4, 2, 22, 64, "e4m3")
    q, k, v = (torch.randn(3, h, 64, device="cuda").bfloat16() for h in (4, 2, 2))
    lengths, slots = i32([0, 15, 30]), i32([3, 0, 1])
    c2, s2, l2 = c.clone(), s.clone(), lengths.clone()
    gdn.swa_step(c2, q, k, v, l2, 2, s2, slots)        # warm up on the copy, then start over
    c2, s2 = c.clone(), s.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gdn.swa_step(c, q, k, v, lengths, 2, s, slots)
        lengths.add_(1)
    for t in range(12):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=torch.Generator("cuda").manual_seed(t), device="cuda"))
        graph.replay()
        want = gdn.swa_step(c2, q, k, v, l2, 2, s2, slots)
        l2 += 1
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(c.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(s, s2)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: the last slots."""
    P, window, sinks = 40, 16380, 4
    c = torch.empty(2, P, 16, window + sinks, 128, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.randn(2, 30, 16, 128, device="cuda").bfloat16() for _ in range(2))
    slots = i32([P - 1, P - 2])
    gdn.cache_write(c, k, v, i32([0, 0]), sinks, None, slots)
    assert torch.equal(c[0, P - 1, :, :30], k[0].transpose(0, 1)) and torch.equal(c[1, P - 2, :, :30], v[1].transpose(0, 1))
    rk, rv = gdn.cache_read(c, i32([30, 30]), sinks, None, slots, k=torch.empty_like(k), v=torch.empty_like(v))
    assert torch.equal(rk, k) and torch.equal(rv, v)
    q = torch.randn(2, 16, 128, device="cuda").bfloat16()
    o = gdn.swa_step(c, q, k[:, 0].contiguous(), v[:, 0].contiguous(), i32([30, 30]), sinks, None, slots)
    kk, vv = torch.cat([k, k[:, :1]], 1), torch.cat([v, v[:, :1]], 1)
    want, _ = gdn.swa_fwd(q[:, None].contiguous(), kk, vv, window, sinks)
    assert (o.float() - want[:, 0].float()).abs().max() <= 4 * HALF["bf16"] * vv.abs().max()
