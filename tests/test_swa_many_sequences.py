"""Windowed attention over as many short sequences as a packed batch may hold: more blocks than one dimension of a launch
counts."""
import pytest
import torch

import gated_delta_rule_24_amd as gdn

from .op_util import U

pytestmark = pytest.mark.gpu


def test_more_blocks_than_a_launch_counts():
    """2^20 sequences of one token and 16 heads: 2^24 blocks, of 2^32 threads, and 2^24 (sequence, head) pairs with sinks.  A
    query sees its own key alone: o = v and dv = d_o, bit for bit (a probability of 1 up to 2^-20, rounded to bf16), lse is the
    score, and dq and dk are what dP and D, equal sums of d products, differ by: 2 (d + 2) U of their terms' size."""
    N, H, d = 1 << 20, 16, 32
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v, do = (torch.randn(1, N, H, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    o, lse = gdn.swa_fwd(q, k, v, 1, 1, cu)
    assert torch.equal(o, v)
    s = (q.float() * k.float()).sum(-1) * d ** -0.5
    size = (q.float() * k.float()).abs().sum(-1) * d ** -0.5
    assert ((lse - s).abs() <= (2 * d + 16) * U * size).all()
    dq, dk, dv = gdn.swa_bwd(do, q, k, v, o, lse, 1, 1, cu)
    assert torch.equal(dv, do)
    room = 2 * (d + 2) * U * (do.float() * v.float()).abs().sum(-1, keepdim=True) * d ** -0.5
    for got, by in ((dq, k), (dk, q)):
        assert (got.float().abs() <= 1.01 * room * by.float().abs()).all()
