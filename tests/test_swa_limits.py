"""Windowed attention where sizes pass what a number or a launch holds: offsets past 32 bits, several thousand
sequences, units shared out over the GPU's parts, windows and masks at their ends."""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn

from .op_util import HALF, cu_tensor, dev
from .test_swa import check as check_fwd
from .test_swa import inputs
from .test_swa_bwd import check as check_bwd

pytestmark = pytest.mark.gpu


def test_offsets_past_32_bits():
    """Tensors of 4.6 GB.  The last rows see the sinks and the rows before them alone, so that they and what they give
    back are those of a short call on the sinks and the last rows, up to the order of the sums: two roundings of
    the operands and one of the result on each side, 6 half steps of the largest term, and as many terms as rows see."""
    T, H, d, window, sinks, tail = 1_120_000, 16, 128, 12, 2, 100
    g = torch.Generator("cuda").manual_seed(1)
    new = lambda: torch.randn(1, T, H, d, generator=g, device="cuda", dtype=torch.bfloat16)     # noqa: E731
    q, k, v, do = new(), new(), new(), new()
    assert q.numel() * 2 > 2 ** 32
    o, lse = gdn.swa_fwd(q, k, v, window, sinks)
    dq, dk, dv = gdn.swa_bwd(do, q, k, v, o, lse, window, sinks)
    last = lambda x, n: x[:, T - n:].contiguous()                                               # noqa: E731
    few = lambda x: torch.cat([x[:, :sinks], x[:, T - tail:]], 1)                               # noqa: E731
    so, slse = gdn.swa_fwd(last(q, tail), few(k), few(v), window, sinks)
    sq, sk, sv = gdn.swa_bwd(last(do, tail), last(q, tail), few(k), few(v), so, slse, window, sinks)
    n, h = 60, HALF["bf16"]
    big = [x.float().abs().max().item() for x in (last(q, tail), few(k), few(v), last(do, tail))]
    pairs = ((last(o, n), so[:, -n:], big[2]),
             (last(dq, n), sq[:, -n:], 2 * d ** 0.5 * big[2] * big[3] * big[1]),
             (last(dk, n), sk[:, -n:], 2 * d ** 0.5 * big[2] * big[3] * big[0] * window),
             (last(dv, n), sv[:, -n:], big[3] * window))
    for got, want, size in pairs:
        assert (got.float() - want.float()).abs().max().item() <= 6 * h * size
    assert (last(lse, n) - slse[:, -n:]).abs().max().item() <= 1e-5
    assert all(x[:, T // 2].float().abs().sum() > 0 for x in (o, dq, dk, dv))


def test_gradient_of_many_sequences():
    """More sequences than the table kernel has threads, empty ones among them."""
    lens = np.random.default_rng(8).integers(0, 4, 2500)
    cu = [0] + np.cumsum(lens).tolist()
    t, x = inputs(8, 1, cu[-1], cu[-1], 2, 1, 32, "fp32")
    check_bwd(t, x, "fp32", 2, 1, cu, label="2500 sequences")


@pytest.mark.parametrize("B,H,KV,d", [(4, 4, 2, 32), (8, 3, 1, 64), (1, 16, 8, 32), (2, 4, 4, 128)])
def test_pairs_shared_out_evenly(B, H, KV, d):
    """As many (sequence, key head) pairs as the GPU's eight parts divide: units in another order, far parts too."""
    t, x = inputs(B, B, 400, 400, H, KV, d, "bf16")
    check_fwd(t, x, "bf16", 30, 3, label=f"pairs {B} x {KV}")
    check_bwd(t, x, "bf16", 30, 3, label=f"pairs {B} x {KV}")


@pytest.mark.parametrize("window", [1, 127, 128, 129, 2 ** 31 - 1, 2 ** 40])
def test_windows_at_their_ends(window):
    t, x = inputs(3, 1, 260, 260, 2, 1, 32, "fp32")
    check_fwd(t, x, "fp32", window, 0, label=f"window {window}")
    check_bwd(t, x, "fp32", window, 128, label=f"window {window}, 128 sinks")


def test_binding_refuses_numbers_that_do_not_fit():
    q = torch.zeros(1, 4, 1, 32, device="cuda")
    for kw in (dict(window=0), dict(window=-2 ** 40), dict(sinks=-1), dict(sinks=129)):
        with pytest.raises(gdn.GdnError):
            gdn.swa_fwd(q, q, q, **{"window": 4, **kw})
    with pytest.raises(ValueError):
        gdn.swa_fwd(q, q, q, 4, 2 ** 32)
    with pytest.raises(ValueError):
        gdn.swa_fwd(torch.zeros(1, 4, 2, 32, device="cuda")[:, :, :1], q, q, 4)
    with pytest.raises(ValueError):
        gdn.swa_fwd(q, q.bfloat16(), q, 4)
    with pytest.raises(ValueError):
        gdn.swa_fwd(q, q, q, 4, cu_seqlens_k=cu_tensor([0, 4]))
    cache = torch.zeros(2, 3, 1, 8, 32, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        gdn.swa_step(cache, q[0], q[0], q[0], n)                       # four queries, two lengths
    with pytest.raises(ValueError):
        gdn.cache_write(cache, q, q, n, 8)                             # no room for a window
    with pytest.raises(gdn.GdnError):
        gdn.cache_write(cache, q.bfloat16(), q.bfloat16(), n[:1])


def test_everything_not_finite():
    """Everything NaN: the careful pass over whole tiles ends, and gives NaN where something is seen."""
    t, _ = inputs(5, 1, 300, 300, 2, 1, 64, "bf16")
    bad = [torch.full_like(y, float("nan")) for y in t]
    o, lse = gdn.swa_fwd(*bad, 40, 2)
    assert torch.isnan(o).all() and torch.isnan(lse).all()
    for g in gdn.swa_bwd(bad[0], *bad, o, lse, 40, 2):
        assert torch.isnan(g).all()
    big = [dev(1e30 * np.ones(y.shape), "bf16") for y in t]            # scores that overflow
    o, _ = gdn.swa_fwd(*big, 40, 2)
    assert torch.isnan(o).all()
