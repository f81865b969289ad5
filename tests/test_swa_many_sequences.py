"""Windowed attention over as many short sequences as a packed batch may hold: more blocks than one dimension of a launch
counts, and a workspace for what they need alone."""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn

from .op_util import DT, HALF, U, cu_tensor, host, within
from .swa_terms import gradients
from .test_swa import inputs


def test_workspace_of_short_sequences():
    """Parts of the sinks' gradients are kept for sequences longer than a window and a key tile: for each window + 128
    keys of the batch at most two, whatever the number of sequences."""
    size = gdn.swa_bwd_workspace_size
    for n in (1, 256):
        one = (1, 2386, 2386, 16, 16, 128, n, 2048)
        assert size(*one, 128) - size(*one, 0) < 2 * (2 * 16 * 2 * 128 * 128 * 4)
    assert size(1, 131072, 131072, 32, 32, 32, 131072, 4096, 4) < 131072 * 32 * 4 + (1 << 25)
    long = size(1, 32768, 32768, 16, 8, 64, 1, 2048, 16)                  # parts: 15 slots, twice
    assert 32768 * 16 * 4 + 15 * 8 * 2 * 16 * 64 * 4 < long < 32768 * 16 * 4 + 31 * 8 * 2 * 16 * 64 * 4 + (1 << 16)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,sinks", [("bf16", 64, 3), ("fp32", 32, 128), ("fp16", 128, 1)])
def test_far_parts_side_by_side(dtype, d, sinks):
    """Sequences with none, one and several far parts next to each other, of lengths at their borders, with more keys
    than queries and fewer; in rows as well."""
    window = 9
    far = window + 128
    lens = [(far, far), (far - 1, far - 1), (0, 3 * far), (far + 1, far + 1), (1, 2 * far), (2 * far, 2 * far), (5, 0),
            (0, 0), (3 * far + 5, 3 * far - 4), (40, 2 * far - 1), (far, far)]
    cu, cuk = ([0, *np.cumsum([x[i] for x in lens]).tolist()] for i in (0, 1))
    for B, T, Tk, c, ck in ((1, cu[-1], cuk[-1], cu, cuk), (3, 2 * far + 3, 2 * far + 3, None, None)):
        t, x = inputs(d + B, B, T, Tk, 2, 1, d, dtype)
        do = torch.randn(t[0].shape, generator=torch.Generator("cuda").manual_seed(B), device="cuda").to(DT[dtype])
        o, lse = gdn.swa_fwd(*t, window, sinks, cu_tensor(c), cu_tensor(ck))
        ws = torch.full((gdn.swa_bwd_workspace_size(B, T, Tk, 2, 1, d, B if c is None else len(lens), window, sinks, DT[dtype]),),
                        255, dtype=torch.uint8, device="cuda")            # a part that is read and was not written: NaN
        got = gdn.swa_bwd(do, *t, o, lse, window, sinks, cu_tensor(c), cu_tensor(ck), workspace=ws)
        for name, y, (w, room) in zip(("dq", "dk", "dv"), got, gradients(
                host(do), *x, host(o), host(lse), window, sinks, c, ck, h=HALF[dtype])):
            within(y, w, room, dtype, f"{dtype} B{B} {name}")


@pytest.mark.gpu
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
