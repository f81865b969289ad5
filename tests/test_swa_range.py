"""Windowed attention over the range of its numbers: probabilities and gradients of scores far below the largest of
their row, scores and scales of any size.  Closed forms in 64 bits.

FP16 holds a power of two down to 2^-14 with all its bits.  Operands are taken times a power of two that puts the
largest of a row at 2^14 or above (below 2^16), so what is down to 2^-28 of the largest is rounded once (HALF), and what is
less by at most 2^-25 of that unit, 2^-39 of the largest.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn

from .op_util import HALF, U, within
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
