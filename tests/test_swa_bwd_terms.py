"""Gradients of windowed attention, each element within the room that its own terms give it (swa_terms.py), which a wrong
row, a dropped tile or zeros do not fit; gradients past 32 bits; malformed offsets, with what the outputs held."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn

from .op_util import DT, HALF, U, cu_tensor, host, within
from .swa_terms import gradients
from .test_swa import inputs

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv")


def outside(got, want, room, dtype, label):
    """Some element is not within what within() allows."""
    allowed = room + HALF[dtype] * (np.abs(want) + room)
    assert (np.abs(got - want) > allowed).any(), label


def check(t, x, dtype, window, sinks, cu=None, cuk=None, seed=0, label=""):
    do = torch.randn(t[0].shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(DT[dtype])
    c, ck = cu_tensor(cu), cu_tensor(cuk)
    o, lse = gdn.swa_fwd(*t, window, sinks, c, ck)
    got = gdn.swa_bwd(do, *t, o, lse, window, sinks, c, ck)
    torch.cuda.synchronize()
    for name, y, (w, room) in zip(NAMES, got, gradients(host(do), *x, host(o), host(lse), window, sinks, cu, cuk,
                                                        h=HALF[dtype])):
        within(y, w, room, dtype, f"{label} {name}")
        if x[0].shape[1] > 30 and window > 4:                     # else a gradient may be nothing but rounding
            outside(np.zeros_like(w), w, room, dtype, f"{label} {name}: zeros")
            outside(np.roll(host(y), 1, 1), w, room, dtype, f"{label} {name}: a row on")
            if w.shape[2] > 1:
                outside(np.roll(host(y), 1, 2), w, room, dtype, f"{label} {name}: a head on")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("T,H,KV,window,sinks", [
    (1, 1, 1, 1, 0), (2, 4, 2, 1, 1), (31, 3, 3, 5, 0), (33, 2, 1, 7, 2), (64, 2, 2, 64, 0), (130, 6, 2, 1000, 3),
    (200, 2, 2, 33, 1), (257, 2, 1, 100, 40), (400, 3, 1, 10, 128)])
def test_shapes(dtype, d, T, H, KV, window, sinks):
    t, x = inputs(d + T, 2, T, T, H, KV, d, dtype)
    check(t, x, dtype, window, sinks, label=f"{dtype} d{d} T{T} H{H}/{KV} W{window} S{sinks}")


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp16", 128)])
@pytest.mark.parametrize("group", [1, 3, 4, 5, 7, 8, 12, 16])
def test_groups(group, dtype, d):
    t, x = inputs(group, 1, 150, 150, 2 * group, 2, d, dtype)
    check(t, x, dtype, 40, 2, label=f"group {group}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [32, 128])
def test_packed(dtype, d):
    cu = [0, 0, 1, 66, 66, 67, 300, 300]
    t, x = inputs(5, 1, 300, 300, 4, 2, d, dtype)
    check(t, x, dtype, 70, 2, cu, label="packed")
    check(t, x, dtype, 1 << 30, 0, cu, label="packed causal")
    t, x = inputs(6, 1, 200, 330, 4, 2, d, dtype)
    check(t, x, dtype, 50, 5, [0, 100, 100, 200], [0, 70, 90, 330], label="other keys than queries")


@pytest.mark.parametrize("dtype,sinks,group,d", [("bf16", 1, 2, 32), ("bf16", 128, 1, 128), ("fp16", 33, 3, 64),
                                                 ("fp16", 4, 1, 128), ("fp32", 4, 1, 32)])
def test_far_parts_of_the_sinks(dtype, sinks, group, d):
    t, x = inputs(sinks, 1, 2300, 2300, group, 1, d, dtype)
    check(t, x, dtype, 20, sinks, label=f"far parts, {sinks} sinks")
    check(t, x, dtype, 20, sinks, [0, 1300, 1300, 1340, 2300], label=f"far parts packed, {sinks} sinks")
    t, x = inputs(sinks, 1, 1200, 1500, group, 1, d, dtype)
    check(t, x, dtype, 20, sinks, label="behind keys")


@pytest.mark.parametrize("B,H,KV,d", [(4, 4, 2, 32), (8, 3, 1, 64), (1, 16, 8, 32), (2, 4, 4, 128)])
def test_pairs_shared_out_evenly(B, H, KV, d):
    t, x = inputs(B, B, 400, 400, H, KV, d, "bf16")
    check(t, x, "bf16", 30, 3, label=f"pairs {B} x {KV}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
def test_whole_tiles(dtype, d):
    """A window of many tiles: most are seen whole."""
    t, x = inputs(d, 1, 1500, 1500, 4, 2, d, dtype)
    check(t, x, dtype, 900, 3, label="whole tiles")


def test_gradients_past_32_bits():
    """Tensors of 4.6 GB.  dQ, dK and dV about 2^31 bytes, 2^31 elements and the end, from the rows around them and the sinks;
    the sinks' own gradients, which every query adds to, in 64 bits over all of them."""
    T, H, d, window, sinks, tail = 1_120_000, 16, 128, 12, 2, 100
    g = torch.Generator("cuda").manual_seed(2)
    q, k, v, do = (torch.randn(1, T, H, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    assert q.numel() > 2 ** 31
    o, lse = gdn.swa_fwd(q, k, v, window, sinks)
    got = gdn.swa_bwd(do, q, k, v, o, lse, window, sinks)
    for at in (2 ** 31 // (2 * H * d), 2 ** 31 // (H * d), T - 30):
        a, b = at - tail + 30, at + 30
        near = lambda y: host(y[:, a:b])                                                    # noqa: E731
        few = lambda y: np.concatenate([host(y[:, :sinks]), host(y[:, a:b])], 1)            # noqa: E731
        want = gradients(near(do), near(q), few(k), few(v), near(o), near(lse), window, sinks, h=HALF["bf16"])
        for name, y, (w, room), skip in zip(NAMES, got, want, (0, sinks, sinks)):
            rows = slice(window, tail - window if b < T else tail)        # what they see, and what sees them, is here
            w, room = (z[:, skip:][:, rows] for z in (w, room))
            y = y[:, a:b][:, rows]
            within(y, w, room, "bf16", f"{name} about row {at}")
            outside(np.roll(host(y), 1, 1), w, room, "bf16", f"{name}: a row on")
    sums = [torch.zeros(sinks, H, d, dtype=torch.float64, device="cuda") for _ in range(4)]   # dk, dv, their squares
    K, V = k[0, :sinks].double(), v[0, :sinks].double()
    for a in range(0, T, 20_000):
        Q, O, G = (y[0, a:a + 20_000].double() for y in (q, o, do))
        D = (O * G).sum(-1)
        for j in range(sinks):
            p = torch.exp((Q * K[j]).sum(-1) * d ** -0.5 - lse[0, a:a + 20_000].double())
            if a == 0:
                p[:j] = 0.0
            ds = p * ((G * V[j]).sum(-1) - D)
            for i, (w, y) in enumerate(((ds, Q * d ** -0.5), (p, G))):
                sums[i][j] += (w[..., None] * y).sum(0)
                sums[2 + i][j] += ((w[..., None] * y) ** 2).sum(0)
    # an operand's half step, and fp32's (2 d + 40) U of the rest: six times the root of the sum of squares, as in
    # swa_terms.py; sums of at most T / 140 parts
    h = HALF["bf16"] / 3 ** 0.5 + 64 * (2 * d + 40) * U
    for i, name in ((0, "dk"), (1, "dv")):
        within(got[1 + i][0, :sinks], host(sums[i]), 6 * h * np.sqrt(host(sums[2 + i])), "bf16", f"{name} of the sinks")


BAD = [([1, 50, 100], [0, 50, 100], 1), ([0, 60, 50, 100], [0, 50, 60, 100], 2), ([0, 50, 99], [0, 50, 100], 3),
       ([0, 50, 100], [2, 50, 100], 4), ([0, 50, 60, 100], [0, 60, 50, 100], 5), ([0, 50, 100], [0, 50, 101], 6)]


@pytest.mark.parametrize("cu,cuk,code", BAD)
def test_malformed_offsets_leave_the_outputs(cu, cuk, code):
    lib = gdn.load()
    t, _ = inputs(4, 1, 100, 100, 2, 1, 32, "bf16")
    o, lse = gdn.swa_fwd(*t, 10, 1)
    desc = gdn.SwaDesc(1, 100, 100, 2, 1, 32, len(cu) - 1, 10, 1, 1, 0.2, 0)
    c, ck = cu_tensor(cu), cu_tensor(cuk)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    p = lambda y: ctypes.c_void_p(y.data_ptr())                                             # noqa: E731
    outs = [torch.full_like(y, 7.0) for y in (t[0], t[1], t[2], t[0], lse)]
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.gdn_swa_bwd(desc, p(t[0]), *map(p, t), p(o), p(lse), p(c), p(ck), *map(p, outs[:3]), p(ws), 1 << 20,
                           stream) == 0
    assert gdn.chunk_fwd_check(ws) == code
    assert lib.gdn_swa_fwd(desc, *map(p, t), p(c), p(ck), p(outs[3]), p(outs[4]), p(ws), 1 << 20, stream) == 0
    assert gdn.chunk_fwd_check(ws) == code
    assert all((y == 7.0).all() for y in outs)
