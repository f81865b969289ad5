"""Windowed attention over the range of its numbers: probabilities and gradients of scores far below the largest of
their row, scores and scales of any size.  Closed forms in 64 bits.

FP16 holds numbers down to 2^-14 with all their bits.  Operands are taken times a power of two that puts the largest
probability of a row at 2^14 or above, the largest gradient of a score at 2^12 or above (below 2^16), so what is down to
2^-28 (2^-26) of the largest is rounded once (HALF), and what is less is off by 2^-25 at most: 2^-39 (2^-37) of it.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn
from oracle import attention as A

from .op_util import DT, HALF, TINY, U, cu_tensor, host, within
from .swa_terms import gradients
from .test_swa import errors, inputs
from .test_swa_small_weights import bound, case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gap", [*np.arange(14.5, 19.5, 0.5).tolist()])
@pytest.mark.parametrize("n", [2000, 33])
def test_forward_far_below_the_largest(dtype, gap, n):
    """2^-28 is 19.4 nats: one rounding of each probability."""
    (q, k, v), want = case(n, 64, gap, 512.0, dtype)
    o, lse = gdn.swa_fwd(q, k, v, n + 1, scale=1.0)
    within(o, np.full(o.shape, want), bound(n, dtype, want), dtype, f"{dtype} gap {gap}")
    assert abs(lse.item() - (gap + np.log1p(n * np.exp(-gap)))) <= (n + 72) * U + 8 * U * gap


@pytest.mark.parametrize("gap", [20, 22, 24, 26])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_forward_below_that(gap, d):
    """FP16: each of n keys is off by 2^-39 of the largest probability, times its value."""
    n, value = 20000, 512.0
    (q, k, v), want = case(n, d, gap, value, "fp16")
    o, _ = gdn.swa_fwd(q, k, v, n + 1, scale=1.0)
    within(o, np.full(o.shape, want), bound(n, "fp16", want) + n * value * 2.0 ** -39, "fp16", f"d{d} gap {gap}")


@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_forward_maxima_that_move(dtype, order):
    """The largest score so far grows from tile to tile, by less and by more than the distance at which it is followed.
    Values are positive: each probability is rounded once, relative, and a sum's parts are rescaled at most
    once a tile of 32 keys: (n + 72 + 2 n / 32) U + 2 HALF."""
    n, d = 640, 64
    s = {"up": np.arange(n) / 64.0, "down": np.arange(n)[::-1] / 64.0,
         "mixed": np.random.default_rng(2).integers(0, 640, n) / 64.0}[order]
    q, k, v = (torch.zeros(1, t, 1, d, device="cuda") for t in (1, n, n))
    q[..., 0], q[..., 1] = 1.0, 1.0
    k[0, :, 0, 0], k[0, :, 0, 1] = torch.from_numpy(np.floor(s)), torch.from_numpy(s - np.floor(s))   # exact in 8 bits
    value = 1.0 + np.arange(n) % 8 / 8.0
    v[0, :, 0] = torch.from_numpy(value)[:, None]
    q, k, v = (x.to(torch.bfloat16 if dtype == "bf16" else torch.float16 if dtype == "fp16" else torch.float32)
               for x in (q, k, v))
    o, lse = gdn.swa_fwd(q, k, v, n, scale=1.0)
    w = np.exp(s - s.max())
    want = (w * value).sum() / w.sum()
    within(o, np.full(o.shape, want), ((n + 72 + n / 16) * U + 2 * HALF[dtype]) * want, dtype, f"{dtype} {order}")
    assert abs(lse.item() - (s.max() + np.log(w.sum()))) <= (n + 72) * U + 8 * U * 10


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("sinks", [0, 40])
@pytest.mark.parametrize("size", [2.0 ** -10, 2.0 ** -4, 2.0 ** 10])
def test_gradient_of_small_scores(dtype, d, sinks, size):
    """dQ and dK where d_o reaches many small probabilities alone.  One query of the last has a gradient, in column 0,
    where the small keys' values are 1 and the large key's is 0:  dS_j = p_j (size - D),  dS_0 = -p_0 D,  D = size o.
    Column 2 of the small keys makes dQ, column 1 of the query dK; neither is in a score.  The terms have one sign: one rounding
    of dS, and one of o in D: bound()."""
    n, gap, big = 511, 14.0, 2.0 ** 14
    (q, k, v), _ = case(n, d, gap, 1.0, dtype)
    q = q.expand(1, n + 1, 1, d).contiguous()
    q[..., 1], k[:, 1:, :, 2], v[..., 1:] = big, big, 0.0
    do = torch.zeros_like(q)
    do[:, -1, :, 0] = size
    window = 100 if sinks else n + 1
    o, lse = gdn.swa_fwd(q, k, v, window, sinks, scale=1.0)
    dq, dk, _ = gdn.swa_bwd(do, q, k, v, o, lse, window, sinks, scale=1.0)
    seen = [j for j in range(1, n + 1) if n - j < window or j < sinks]
    large = 1.0 if sinks or window > n else 0.0                  # whether the last query sees key 0
    w = np.exp(-gap)
    m = len(seen)
    total = large + m * w
    D = size * m * w / total
    ds = w / total * (size - D)
    label = f"{dtype} d{d} sinks {sinks} size {size}"
    within(dq[0, -1, 0, 2:3], np.array([m * ds * big]), bound(n, dtype, m * ds * big), dtype, f"{label} dq")
    within(dk[0, seen, 0, 1], np.full(m, ds * big), bound(n, dtype, ds * big), dtype, f"{label} dk")
    within(dk[0, :1, 0, 1], np.array([-D * large / total * big]), bound(n, dtype, D * big), dtype, f"{label} dk of the large")
    hidden = [j for j in range(1, n + 1) if j not in seen]
    assert not dk[0, hidden].any() and not dq[0, :-1].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_gradient_of_large_scores(dtype, d):
    """dS past 65504, with results that the type holds: all exact."""
    q, k, v = (torch.zeros(1, 2, 1, d, device="cuda", dtype=x.dtype) for x in case(1, d, 1, 1.0, dtype)[0])
    q[..., 1], k[0, 0, 0, 2], k[0, 1, 0, 2], v[0, 0, 0, 0], v[0, 1, 0, 0] = 2.0 ** -6, 2.0 ** -6, -2.0 ** -6, 4.0, -4.0
    do = torch.zeros_like(q)
    do[0, 1, 0, 0] = 2.0 ** 15
    o, lse = gdn.swa_fwd(q, k, v, 2, scale=1.0)
    dq, dk, dv = gdn.swa_bwd(do, q, k, v, o, lse, 2, scale=1.0)
    # p = 1/2 twice up to the rounding of lse: 4 U
    for got, want in ((dq[0, 1, 0, 2], 2.0 ** 11), (dk[0, 0, 0, 1], 2.0 ** 10), (dk[0, 1, 0, 1], -2.0 ** 10),
                      (dv[0, 0, 0, 0], 2.0 ** 14), (dv[0, 1, 0, 0], 2.0 ** 14)):
        within(got, np.array(want), 8 * U * abs(want), dtype, f"{dtype} d{d}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,keys,size", [(128, 32768, 2.0 ** -6), (128, 32768, 2.0 ** -10), (64, 32768, 2.0 ** -10),
                                         (32, 8192, 2.0 ** -12), (64, 8192, 2.0 ** 6)])
def test_gradient_over_many_keys(dtype, d, keys, size):
    """Some queries that see all of many keys, and gradients of the size that training meets in fp16.  Element by element,
    and by root mean square: two roundings, of dS and of the result, at most HALF / sqrt 3 each, and the fp16 result's
    subnormal step."""
    T, H = 48, 2
    t, x = inputs(d + keys, 1, T, keys, H, 1, d, dtype)
    do = (torch.randn(1, T, H, d, generator=torch.Generator("cuda").manual_seed(7), device="cuda") * size).to(t[0].dtype)
    o, lse = gdn.swa_fwd(*t, keys)
    got = gdn.swa_bwd(do, *t, o, lse, keys)
    want = gradients(host(do), *x, host(o), host(lse), keys, h=HALF[dtype])
    for name, g, (w, room) in zip(("dq", "dk", "dv"), got, want):
        within(g, w, room, dtype, f"{dtype} d{d} {keys} keys {size} {name}")
        off, rms = (np.sqrt(np.mean(y ** 2)) for y in (host(g) - w, w))
        assert off <= HALF[dtype] * rms + TINY[dtype] / 2, (name, off / rms)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("at", [0, 40, 690])
def test_step_beside_an_outlying_scale(dtype, d, at):
    """8-bit rows whose scale is 2^-14, and one of scale 2^20 that hardly counts, in a column of its own, first, among
    them or last.  The weights (probability times scale) have their own largest, e^-40 2^20 or 2^-14: no row's rounding is
    more than HALF of what it adds, and the terms have one sign."""
    if dtype == "fp32" and d == 256:
        pytest.skip("fp32 is built to 128")
    n = 700
    g = np.random.default_rng(at)
    value = g.integers(8, 16, n) / 8.0                           # e4m3 holds these
    c = torch.zeros(2, 1, 1, n, d, device="cuda")
    s = torch.ones(2, 1, 1, n, device="cuda")
    c[0, 0, 0, :, 0] = 0.9375                                    # e^-2.5 of a few rows', no power of two
    c[0, 0, 0, 3::16, 0] = 1.0
    s[0, 0, 0, :] = torch.where(torch.arange(n, device="cuda") == at, 2.0 ** -60, 1.0)    # its score is 0
    c[1, 0, 0, :, 0] = torch.from_numpy(value)
    c[1, 0, 0, at] = 0.0
    c[1, 0, 0, at, d - 1] = 1.5
    s[1, 0, 0, :] = torch.where(torch.arange(n, device="cuda") == at, 2.0 ** 20, 2.0 ** -14)
    q = torch.zeros(1, 1, d, dtype=DT[dtype], device="cuda")
    q[..., 0] = 40.0
    score = 40.0 * host(c)[0, 0, 0, :, 0] * host(s)[0, 0, 0]
    new = torch.zeros(1, 1, d, dtype=DT[dtype], device="cuda")
    new[..., 0] = 1.0                                            # the row that is written: score 40
    o = gdn.swa_step(c.to(torch.float8_e4m3fn), q, new, new * 2.0 ** -14, torch.full((1,), n - 1, dtype=torch.int32, device="cuda"),
                     0, s, scale=1.0)
    score[-1] = 40.0
    w = np.exp(score - 40.0)
    v = host(c)[1, 0, 0] * host(s)[1, 0, 0][:, None]
    v[-1] = 0.0
    v[-1, 0] = 2.0 ** -14
    want = (w @ v) / w.sum()
    within(o[0, 0], want, bound(n, dtype, want), dtype, f"{dtype} d{d} at {at}")


def large(dtype, d, size, sign, n):
    """n keys whose scores are sign size - step j, exact in fp32, and the values: (q, k, v, scores)."""
    step = max(1.0, size * 2.0 ** -23)
    a = 2.0 ** (np.log2(size) // 2)
    q, k, v = (torch.zeros(1, t, 1, d, device="cuda") for t in (1, n, n))
    q[..., 0], q[..., 1] = a, 2.0 ** (np.log2(step) // 2)
    k[..., 0] = sign * size / a
    k[0, :, 0, 1] = -torch.arange(n, device="cuda") % 7 * (step / 2.0 ** (np.log2(step) // 2))
    g = np.random.default_rng(n)
    v[0, :, 0] = torch.from_numpy(g.uniform(0.5, 2.0, (n, d)))
    q, k, v = (x.to(DT[dtype]) for x in (q, k, v))
    return q, k, v, host(k)[0, :, 0] @ host(q)[0, 0, 0]


LARGE = [(2.0 ** 16, "fp16"), (2.0 ** 20, "fp16"), (2.0 ** 24, "fp16"), (2.0 ** 25, "fp16"), (2.0 ** 26, "fp16"),
         (2.0 ** 27, "fp16"), (2.0 ** 28, "fp16"), (2.0 ** 29, "fp16"), (2.0 ** 20, "bf16"), (2.0 ** 26, "bf16"),
         (2.0 ** 31, "bf16"), (2.0 ** 32, "bf16"), (2.0 ** 34, "bf16"), (2.0 ** 40, "bf16"), (2.0 ** 20, "fp32"),
         (2.0 ** 31, "fp32"), (2.0 ** 33, "fp32"), (2.0 ** 60, "fp32")]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size,dtype", LARGE)
@pytest.mark.parametrize("d,n", [(64, 300), (128, 33)])
def test_large_scores(size, dtype, sign, d, n):
    """Scores as large as products of the type are, which fp32 holds exactly, and differ by few of their units: the softmax is of
    the differences.  Its exponents are below 6 size 2^-23 log2 e, off by 2 U of that; past 40 the exponential is below the rest's
    rounding.  lse: two roundings of its size more."""
    q, k, v, s = large(dtype, d, size, sign, n)
    x = s - s.max()
    w = np.exp(x)
    want = (w @ host(v)[0, :, 0]) / w.sum()
    room = 2 * ((n + 72 + 40 * 4) * U + HALF[dtype]) * want
    o, lse = gdn.swa_fwd(q, k, v, n, scale=1.0)
    within(o[0, 0, 0], want, room, dtype, f"{dtype} d{d} {sign * size}")
    assert abs(lse.item() - (s.max() + np.log(w.sum()))) <= 8 * U * size
    c = torch.zeros(2, 1, 1, n, d, device="cuda", dtype=DT[dtype])
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.cache_write(c, k[:, :-1].contiguous(), v[:, :-1].contiguous(), zero)
    o = gdn.swa_step(c, q[:, 0], k[:, -1], v[:, -1], zero + n - 1, scale=1.0)
    within(o[0, 0], want, room, dtype, f"step {dtype} d{d} {sign * size}")


def test_large_scores_beside_small_ones():
    """Rows of either kind in one tile, in packed sequences, with sinks and hidden values that are not finite."""
    T, d = 200, 64
    t, x = inputs(77, 1, T, T, 2, 1, d, "fp32")
    t[0][0, 50:60] *= 2.0 ** 24
    t[0][0, 130] *= -2.0 ** 33
    cu = [0, 90, 200]
    o, lse = gdn.swa_fwd(*t, 30, 2, cu_tensor(cu))
    q, k, v = (host(y) for y in t)
    # fp32's scores themselves are off: those rows by what their own scores say, the others as ever
    calm = np.ones(T, bool)
    calm[50:60] = calm[130] = False
    ro, rl = A.attention(q, k, v, 30, 2, cu)
    within(o[0, calm], ro[0, calm], 2 * (errors(q[0, calm], k, d ** -0.5) + 200 * U) * np.abs(v).max(), "fp32", "calm rows")
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    seen = [90, 91, *range(101, 131)]                            # one key takes all of row 130
    best = seen[int(np.argmax(q[0, 130, 0] @ k[0, seen, 0].T))]
    within(o[0, 130, 0], v[0, best, 0], 0.0, "fp32", "one key")
    v2 = t[2].clone()
    v2[0, 150:] = float("nan")
    again, _ = gdn.swa_fwd(t[0], t[1], v2, 30, 2, cu_tensor(cu))
    within(again[0, :150], host(o)[0, :150], 64 * U * np.abs(v).max(), "fp32", "hidden values")
