"""The gated linear recurrence at the limits of its values and sizes."""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn
from oracle import operators as R

from .op_util import DT, cu_tensor, dev, host

pytestmark = pytest.mark.gpu

INF = float("inf")


def same(got, want, clean, label):
    """Not-a-number and infinities where the fp64 recurrence has them, elsewhere the bits of `clean`."""
    g = host(got)
    assert np.array_equal(np.isnan(g), np.isnan(want)), label
    assert np.array_equal(np.where(np.isinf(g), g, 0), np.where(np.isinf(want), want, 0)), label
    finite = torch.from_numpy(np.isfinite(want)).cuda()
    assert torch.equal(got[finite], clean[finite]), label


@pytest.mark.parametrize("patience", ["4096", "0"])
@pytest.mark.parametrize("gate", [-0.05, -1.0, -20.0])
@pytest.mark.parametrize("gate_type", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,D,cu", [(20, 8, None), (100, 3, None), (9000, 3, None), (9000, 24, None),
                                    (9000, 3, [0, 40, 40, 8800, 9000]), (9000, 24, [0, 40, 40, 8800, 9000])])
def test_infinite_states_decay_as_the_recurrence_says(monkeypatch, T, D, cu, gate_type, gate, patience):
    """An infinite state times decays that are not 0 is infinite, whatever the product of the decays is in fp32
    (-0.05 underflows over a few tiles of 128 tokens, -1 within a tile, -20 within a thread's 8 tokens); times a
    decay of 0 it is not-a-number.  One channel each: an infinite initial state, an infinite x in the middle, both
    with a decay of 0 later on, where there are channels for it."""
    monkeypatch.setenv("GDN_SCAN_PATIENCE", patience)
    g = np.random.default_rng(T + D)
    N = 1 if cu is None else len(cu) - 1
    at, end = (T // 3, T - 2) if cu is None else (3000, 8000)     # both in the long sequence
    n = 0 if cu is None else 2
    x, dh = g.standard_normal((1, T, D)), g.standard_normal((1, T, D))
    la = np.full((1, T, D), gate)
    init, dfin = g.standard_normal((N, D)), g.standard_normal((N, D))
    put = lambda *v: [dev(u, gate_type if i == 1 else "fp32") for i, u in enumerate(v)]    # noqa: E731
    clean = put(x, la, init, dh, dfin)
    init[n, 0], x[0, at, 1] = INF, -INF
    dfin[n, 0], dh[0, end, 1] = -INF, INF
    if D > 4:
        init[n, 4], dfin[n, 4] = -INF, INF
        la[0, (at + end) // 2, 4] = -INF
        x[0, at, 5], x[0, at + 5, 5] = INF, -INF                  # infinities of both signs meet
        dh[0, end, 5], dh[0, end - 3, 5] = INF, -INF
    t = put(x, la, init, dh, dfin)
    cuts = cu_tensor(cu)
    h, fin = gdn.scan_fwd(t[0], t[1], t[2], cuts)
    ch, cfin = gdn.scan_fwd(clean[0], t[1], clean[2], cuts)
    with np.errstate(invalid="ignore"):
        want, wfin = R.scan(*(host(v) for v in t[:3]), cu)
        wx, wl, wi = R.scan_bwd(host(t[1]), host(ch), host(t[3]), host(clean[2]), host(t[4]), cu)
    assert np.isinf(want).any() and np.isinf(wx).any()
    same(h, want, ch, "h")
    same(fin, wfin, cfin, "final state")
    dx, dl, di = gdn.scan_bwd(t[1], ch, t[3], clean[2], t[4], cuts)
    cx, cl, ci = gdn.scan_bwd(t[1], ch, clean[3], clean[2], clean[4], cuts)
    same(dx, wx, cx, "dx")
    same(dl, wl, cl, "dlog_alpha")
    same(di, wi, ci, "d_init")


@pytest.mark.parametrize("bits", [0x7FC00000, 0xFFC00000, 0xFFFFFFFF], ids=hex)
@pytest.mark.parametrize("gate_type", ["fp32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 5, 60, 2000, 2000, 2300], None], ids=str)
def test_gates_that_are_not_a_number(cu, gate_type, bits):
    """Not-a-number of either sign as a gate: everything behind it in its channel and sequence is not-a-number
    (before it, for the gradient), over several tiles, and nothing else changes."""
    T, D, t0 = 2300, 40, 300
    g = torch.Generator(device="cuda").manual_seed(5)
    x, d = (torch.randn(1, T, D, generator=g, device="cuda") for _ in range(2))
    la = (-torch.rand(1, T, D, generator=g, device="cuda")).to(DT[gate_type])
    cuts, (first, end), n = cu_tensor(cu), ((60, 2000) if cu else (0, T)), 2 if cu else 0
    clean = gdn.scan_fwd(x, la, None, cuts)
    cgrad = gdn.scan_bwd(la, clean[0], d, None, None, cuts)
    bad = la.clone()
    raw = bad.view(torch.int32 if gate_type == "fp32" else torch.int16)
    raw[0, t0, 7] = np.array([bits >> (0 if gate_type == "fp32" else 16)], dtype=np.uint32).astype(
        np.uint32 if gate_type == "fp32" else np.uint16).view(np.int32 if gate_type == "fp32" else np.int16)[0].item()
    h, fin = gdn.scan_fwd(x, bad, None, cuts)
    dx, dl, di = gdn.scan_bwd(bad, clean[0], d, None, None, cuts)
    assert h[0, t0:end, 7].isnan().all() and fin[n, 7].isnan()
    assert dx[0, first:t0, 7].isnan().all() and dl[0, first + 1:t0 + 1, 7].isnan().all() and di[n, 7].isnan()
    h[0, t0:end, 7], fin[n, 7] = clean[0][0, t0:end, 7], clean[1][n, 7]
    dx[0, first:t0, 7], dl[0, first:t0 + 1, 7], di[n, 7] = cgrad[0][0, first:t0, 7], cgrad[1][0, first:t0 + 1, 7], \
        cgrad[2][n, 7]
    for got, want in ((h, clean[0]), (fin, clean[1]), (dx, cgrad[0]), (dl, cgrad[1]), (di, cgrad[2])):
        assert torch.equal(got, want)


def test_decays_below_the_smallest_normal_number_are_zero():
    """alpha has no values between 0 and 2^-126: at log_alpha = -90 a finite state is forgotten, in every form."""
    x = torch.randn(2, 300, 20, device="cuda")
    la = torch.full_like(x, -90.0)
    init = 1e30 * torch.randn(2, 20, device="cuda")
    h, fin = gdn.scan_fwd(x, la, init)
    assert torch.equal(h, x) and torch.equal(fin, x[:, -1])
    assert torch.equal(gdn.scan_fwd(x[:, :5].contiguous(), la[:, :5].contiguous(), init)[0], x[:, :5])
    assert torch.equal(gdn.scan_step(init.clone(), x[:, 0].contiguous(), la[:, 0].contiguous()), x[:, 0])


@pytest.mark.parametrize("gate_type,some,zero", [("fp32", -87.3, -87.4), ("bf16", -87.0, -87.5),
                                                 ("fp16", -87.3125, -87.375)])
@pytest.mark.parametrize("T", [1, 5, 300, 9000])
def test_the_border_of_zero_decays(T, gate_type, some, zero):
    """The last log_alpha whose decay is not 0 and the first whose decay is, by what they make of an infinite state
    in each kernel: infinite and not-a-number."""
    x = torch.randn(1, T, 8, device="cuda")
    init = torch.full((1, 8), INF, device="cuda")
    for gate, test in ((some, torch.isinf), (zero, torch.isnan)):
        la = torch.full((1, T, 8), gate, device="cuda").to(DT[gate_type])
        h, fin = gdn.scan_fwd(x, la, init)
        assert test(h).all() and test(fin).all()
        assert test(gdn.scan_step(init.clone(), x[:, 0].contiguous(), la[:, 0].contiguous())).all()
        dx, _, di = gdn.scan_bwd(la, torch.zeros_like(x), x, None, init)
        assert torch.isinf(dx[:, -1]).all() and test(dx[:, :-1]).all() and test(di).all()


@pytest.mark.parametrize("N,T,D", [(5000, 16, 40), (3000, 1, 3), (70_000, 300, 5), (2500, 0, 16)])
def test_many_empty_sequences(N, T, D):
    """More sequences than blocks and tokens: empty ones hand on what they were given, in place and elsewhere."""
    g = np.random.default_rng(N)
    cu = np.concatenate([[0], np.sort(g.integers(0, T + 1, N - 1)), [T]]).tolist()
    x, d, init, dfin = (dev(g.standard_normal(s)) for s in ((1, T, D), (1, T, D), (N, D), (N, D)))
    la, cuts = -x.abs(), cu_tensor(cu)
    empty = torch.tensor(np.diff(cu) == 0).cuda()
    h, fin = gdn.scan_fwd(x, la, init, cuts)
    assert torch.equal(fin[empty], init[empty])
    assert not gdn.scan_fwd(x, la, None, cuts)[1][empty].any()
    state = init.clone()
    h2, _ = gdn.scan_fwd(x, la, state, cuts, final_state=state)
    assert torch.equal(h, h2) and torch.equal(state, fin)
    for n in np.flatnonzero(np.diff(cu))[:5]:          # the others are as they are alone
        t = slice(cu[n], cu[n + 1])
        alone = gdn.scan_fwd(x[:, t].clone(), la[:, t].clone(), init[n:n + 1].clone())
        assert torch.allclose(fin[n], alone[1][0], rtol=1e-5, atol=1e-6)
    di = gdn.scan_bwd(la, h, d, init, dfin, cuts)[2]
    assert torch.equal(di[empty], dfin[empty])
    assert not gdn.scan_bwd(la, h, d, init, None, cuts)[2][empty].any()


def test_more_tiles_than_one_grid_dimension():
    """Over 2^20 tiles: the last rows are those of a small call, and of the oracle's."""
    B, T = 1_100_000, 33
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(B, T, 1, generator=g, device="cuda")
    la = -torch.rand(B, T, 1, generator=g, device="cuda")
    d = torch.randn(B, T, 1, generator=g, device="cuda")
    h, fin = gdn.scan_fwd(x, la)
    grads = gdn.scan_bwd(la, h, d)
    for part in (slice(0, 40), slice((1 << 20) - 20, (1 << 20) + 20), slice(B - 40, B)):
        sx, sl, sd = (v[part].contiguous() for v in (x, la, d))
        sh, sf = gdn.scan_fwd(sx, sl)
        assert torch.equal(h[part], sh) and torch.equal(fin[part], sf)
        # 33 terms, each off by at most 8 + 4 |l| steps of fp32 a decay: 33 (12 * 33 + 40) 2^-24 of 33 values
        assert np.abs(host(sh) - R.scan(host(sx), host(sl))[0]).max() <= 33 * 440 * 2.0 ** -24 * float(sx.abs().max())
        small = gdn.scan_bwd(sl, sh, sd)
        assert torch.equal(grads[0][part], small[0]) and torch.equal(grads[1][part], small[1])
        assert torch.equal(grads[2][part], small[2])
