"""Windowed attention where one key takes nearly all of the softmax and adds nothing, so that the output is the sum of
many small probabilities; and values whose scales in the cache fp16 does not hold.

All terms of the output have one sign, so its bound is relative.  The small rows' score is 0, and the large
one's exact too; its exponential's argument, below 32 log2(e), is off by less than 64 U.  A
probability is rounded once in the tensors' type, its sum and the products in fp32: (n + 72) U + 2 HALF, and the
rounding of the output."""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn

from .op_util import DT, HALF, U, host, within

pytestmark = pytest.mark.gpu


def case(n, d, gap, value, dtype):
    """n keys of score 0 whose values are `value`, behind one of score `gap` whose value is 0: (q, k, v, o)."""
    q, k, v = (torch.zeros(1, t, 1, d, device="cuda") for t in (1, n + 1, n + 1))
    q[..., 0], k[:, 0, :, 0], v[:, 1:] = 1.0, gap, value
    w = np.exp(-float(gap))
    return [x.to(DT[dtype]) for x in (q, k, v)], value * n * w / (1 + n * w)


def bound(n, dtype, want):
    return ((n + 72) * U + 2 * HALF[dtype]) * want


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gap", [1, 9, 14, 16.25])
@pytest.mark.parametrize("n", [2000, 33])
def test_forward(dtype, gap, n):
    (q, k, v), want = case(n, 64, gap, 512.0, dtype)
    o, lse = gdn.swa_fwd(q, k, v, n + 1, scale=1.0)
    within(o, np.full(o.shape, want), bound(n, dtype, want), dtype, f"{dtype} gap {gap}")
    assert abs(lse.item() - (gap + np.log1p(n * np.exp(-gap)))) <= (n + 72) * U + 8 * U * gap


@pytest.mark.parametrize("kind,dtype", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("e4m3", "bf16"),
                                        ("e4m3", "fp16"), ("e4m3", "fp32")])
@pytest.mark.parametrize("gap,value", [(1, 2.0 ** -10), (6, 2.0 ** -9), (14, 512.0), (16.25, 512.0)])
@pytest.mark.parametrize("n", [2000, 33])
def test_step(kind, dtype, gap, value, n):
    (q, k, v), want = case(n, 64, gap, value, dtype)
    c = torch.zeros(2, 1, 1, n + 1, 64, device="cuda").to(torch.float8_e4m3fn if kind == "e4m3" else DT[kind])
    s = torch.ones(2, 1, 1, n + 1, device="cuda") if kind == "e4m3" else None
    gdn.cache_write(c, k[:, :n].contiguous(), v[:, :n].contiguous(), torch.zeros(1, dtype=torch.int32, device="cuda"),
                    0, s)
    o = gdn.swa_step(c, q[:, 0], k[:, n], v[:, n], torch.full((1,), n, dtype=torch.int32, device="cuda"), 0, s,
                     scale=1.0)
    # an 8-bit key is rounded as it is written
    if kind == "e4m3":
        held = host(c.float())[0, 0, 0, 0, 0] * host(s)[0, 0, 0, 0]
        want = case(n, 64, held, value, dtype)[1]
    within(o, np.full(o.shape, want), bound(n, dtype, want), dtype, f"{kind} {dtype} gap {gap}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_values_of_any_size_in_turn(dtype):
    """Scales of an 8-bit cache from tile to tile larger, smaller and past fp16's range, each row weighted alike."""
    n, d = 700, 64
    size = 2.0 ** np.resize([-30, -9, 3, -20, 6, -12, 0], n // 32 + 1).repeat(32)[:n]
    c = torch.ones(2, 1, 1, n, d, device="cuda").to(torch.float8_e4m3fn)
    s = torch.from_numpy(np.stack([np.ones(n), size]).astype(np.float32)).cuda().view(2, 1, 1, n)
    q = torch.zeros(1, 1, d, dtype=DT[dtype], device="cuda")
    new = torch.full((1, 1, d), 1.0, dtype=DT[dtype], device="cuda")
    o = gdn.swa_step(c, q, new, new, torch.full((1,), n - 1, dtype=torch.int32, device="cuda"), 0, s)
    want = (size[:-1].sum() + 1) / n
    within(o, np.full(o.shape, want), bound(n, dtype, want), dtype, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sinks", [0, 40])
def test_gradient_of_values(dtype, d, sinks):
    """dV of the small keys, p dO: one product of a rounded probability.  512 queries, the last of them with a gradient;
    with sinks the keys before the window are seen too."""
    n, gap, size = 511, 14, 1024.0
    (q, k, v), _ = case(n, d, gap, 512.0, dtype)
    q = q.expand(1, n + 1, 1, d).contiguous()
    do = torch.zeros_like(q)
    do[:, -1] = size
    window = 100 if sinks else n + 1
    o, lse = gdn.swa_fwd(q, k, v, window, sinks, scale=1.0)
    dv = gdn.swa_bwd(do, q, k, v, o, lse, window, sinks, scale=1.0)[2][0, :, 0]
    seen = [j for j in range(1, n + 1) if n - j < window or j < sinks]
    w = np.exp(-float(gap))
    want = size * w / (1 + len(seen) * w)
    within(dv[seen], np.full((len(seen), d), want), bound(n, dtype, want), dtype, f"{dtype} d{d} sinks {sinks}")
    hidden = [j for j in range(1, n + 1) if j not in seen]
    assert not dv[hidden].any()
