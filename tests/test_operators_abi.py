"""Refusals of the gated linear recurrence, layer norm and state move calls:
each returns its status before anything is launched (no GPU needed; the
placeholder pointers are never followed)."""
import ctypes

import pytest
import torch

import gated_delta_rule_24_amd as gdn

A, B, C, D_, E, F = (0x10000000 * i for i in range(1, 7))    # placeholder addresses, 256 MiB apart
WS = 0x100000000


@pytest.fixture(scope="module")
def lib():
    return gdn.load()


def scan_desc(**kw):
    d = dict(batch=2, seqlen=100, channels=96, num_seqs=2, in_dtype=1, gate_dtype=0, out_dtype=1, flags=0)
    d.update(kw)
    return gdn.ScanDesc(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(in_dtype=3), 3), (dict(gate_dtype=-1), 3), (dict(out_dtype=9), 3), (dict(out_dtype=2), 5),
    (dict(batch=0), 2), (dict(seqlen=-1), 2), (dict(channels=0), 2), (dict(num_seqs=0), 2),
    (dict(channels=65537), 5), (dict(flags=1), 5), (dict(batch=1 << 16, seqlen=1 << 14), 2),
])
def test_scan_descriptor(lib, kw, code):
    n = ctypes.c_size_t(0)
    assert lib.gdn_scan_workspace_size(scan_desc(**kw), ctypes.byref(n)) == code
    assert lib.gdn_last_error_message()


def test_scan_workspace(lib):
    n = ctypes.c_size_t(0)
    assert lib.gdn_scan_workspace_size(scan_desc(), ctypes.byref(n)) == 0 and n.value >= 256
    assert lib.gdn_scan_workspace_size(scan_desc(), None) == 1
    assert lib.gdn_scan_workspace_size(None, ctypes.byref(n)) == 1
    assert gdn.scan_workspace_size(1, 50408, 2048, 8) >= 256


def test_scan_fwd_refusals(lib):
    def call(d=None, x=A, la=B, init=None, cu=None, h=C, fin=None, ws=WS, size=1 << 40):
        return lib.gdn_scan_fwd(d or scan_desc(), x, la, init, cu, h, fin, ws, size, None)

    assert call(x=None) == 1 and call(la=None) == 1 and call(h=None) == 1
    assert call(ws=None) == 6 and call(size=8) == 6
    assert call(x=A + 8) == 4 and call(la=B + 4) == 4 and call(h=C + 2) == 4 and call(init=D_ + 8) == 4
    assert call(d=scan_desc(batch=1, num_seqs=2), cu=D_ + 2) == 4
    assert call(cu=D_) == 2                                  # packed with batch 2
    assert call(d=scan_desc(num_seqs=3)) == 2                # rows and sequences differ
    assert call(h=A) == 8 and call(h=A + 16) == 8            # h over x
    assert call(init=D_, fin=D_ + 16) == 8                   # partial overlap of the states
    assert call(fin=C + 64) == 8 and call(fin=B) == 8 and call(ws=A) == 8
    assert b"overlaps" in lib.gdn_last_error_message()


def test_scan_bwd_refusals(lib):
    def call(d=None, la=A, h=B, init=None, cu=None, dh=C, dfin=None, dx=D_, dla=E, di=None, ws=WS, size=1 << 40):
        return lib.gdn_scan_bwd(d or scan_desc(), la, h, init, cu, dh, dfin, dx, dla, di, ws, size, None)

    for name in ("la", "h", "dh", "dx", "dla"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: F + 8}) == 4, name
    assert call(ws=None) == 6 and call(size=8) == 6
    assert call(cu=F) == 2
    assert call(dx=C) == 8                                   # not in place on d_h
    assert call(dla=D_ + 32) == 8 and call(di=D_) == 8 and call(init=F, di=F) == 8


def test_scan_step_refusals(lib):
    def call(N=4, D=96, i=1, g=0, o=1, state=A, x=B, la=C, h=D_):
        return lib.gdn_scan_step(N, D, i, g, o, state, x, la, h, None)

    assert call(i=4) == 3 and call(i=1, g=2) == 5 and call(N=-1) == 2 and call(D=0) == 2 and call(D=70000) == 5
    assert call(state=None) == 1 and call(h=None) == 1 and call(x=B + 2) == 4
    assert call(h=A) == 8 and call(x=A + 16) == 8
    assert call(N=0, state=None) == 0


def test_layernorm_refusals(lib):
    def fwd(rows=10, dim=96, i=1, o=1, eps=1e-5, x=A, w=B, b=C, y=D_, mean=E, rstd=F):
        return lib.gdn_layernorm_fwd(rows, dim, i, o, eps, x, w, b, y, mean, rstd, None)

    assert fwd(i=5) == 3 and fwd(i=1, o=2) == 5
    assert fwd(rows=-1) == 2 and fwd(rows=1 << 31) == 2 and fwd(dim=0) == 2 and fwd(dim=16385) == 5
    for eps in (-1e-5, float("inf"), float("nan")):
        assert fwd(eps=eps) == 5
    assert fwd(x=None) == 1 and fwd(y=None) == 1 and fwd(mean=None) == 1 and fwd(rstd=None) == 1
    assert fwd(x=A + 2) == 4 and fwd(w=B + 4) == 4 and fwd(mean=E + 2) == 4
    assert fwd(y=A) == 8 and fwd(mean=D_) == 8 and fwd(rstd=E + 4) == 8
    assert fwd(rows=0, x=None, y=None) == 0

    def bwd(rows=10, dim=96, i=1, o=1, dy=A, x=B, mean=C, rstd=C + 64, w=None, dx=D_, dw=E, db=F, ws=WS, size=1 << 40):
        return lib.gdn_layernorm_bwd(rows, dim, i, o, dy, x, mean, rstd, w, dx, dw, db, ws, size, None)

    assert bwd(o=7) == 3 and bwd(i=2, o=1) == 5 and bwd(dim=20000) == 5 and bwd(rows=-1) == 2
    assert bwd(ws=None) == 6 and bwd(size=1) == 6
    for name in ("dy", "x", "mean", "rstd", "dx"):
        assert bwd(**{name: None}) == 1, name
    assert bwd(dy=A + 8) == 4 and bwd(rstd=C + 2) == 4 and bwd(dw=E + 8) == 4
    assert bwd(dx=A) == 8 and bwd(dw=D_) == 8 and bwd(db=E) == 8 and bwd(ws=B) == 8
    n = ctypes.c_size_t(0)
    assert lib.gdn_layernorm_bwd_workspace_size(10, 96, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.gdn_layernorm_bwd_workspace_size(10, 0, ctypes.byref(n)) == 2
    assert lib.gdn_layernorm_bwd_workspace_size(10, 96, None) == 1


def test_state_move_refusals(lib):
    def call(layers=2, slots=16, page=4096, moves=4, state=A, src=B, dst=C, status=None):
        return lib.gdn_state_move(layers, slots, page, moves, state, src, dst, status, None)

    assert call(layers=-1) == 2 and call(slots=0) == 2 and call(page=0) == 2 and call(moves=-1) == 2
    assert call(moves=17) == 2                               # more moves than slots
    assert call(slots=65537) == 5 and call(slots=8192, moves=4097) == 5 and call(page=4098) == 5
    assert call(page=1 << 41) == 2 and call(layers=1 << 30, slots=65536, page=1 << 30) == 2
    assert call(state=None) == 1 and call(src=None) == 1 and call(dst=None) == 1
    assert call(state=A + 4) == 4 and call(src=B + 2) == 4 and call(status=D_ + 1) == 4
    assert call(src=A + 64) == 8 and call(status=B + 4) == 8 and call(status=A) == 8
    assert call(moves=0, state=None, src=None, dst=None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 8)
    for f in (lambda: gdn.scan_fwd(x, x), lambda: gdn.scan_bwd(x, x, x), lambda: gdn.scan_step(x[0], x[0], x[0]),
              lambda: gdn.layernorm_fwd(x), lambda: gdn.layernorm_bwd(x, x, x[..., 0], x[..., 0]),
              lambda: gdn.state_move(x, x.int(), x.int())):
        with pytest.raises(ValueError, match="expected a GPU"):
            f()
    with pytest.raises(TypeError):
        gdn.layernorm_fwd([1.0])
