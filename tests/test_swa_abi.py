"""Refusals of the windowed attention and cache calls: each returns its status before
anything is launched (no GPU needed; the placeholder pointers are never followed)."""
import ctypes

import pytest
import torch

import gated_delta_rule_24_amd as gdn

A, B, C, D_, E, F, G, H, I, J, K = (0x100000000 * i for i in range(1, 12))    # placeholder addresses, 4 GiB apart
WS = 0x1000000000
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return gdn.load()


def desc(**kw):
    d = dict(batch=2, seqlen=100, keylen=120, heads=8, kv_heads=2, dim=64, num_seqs=2, window=32, sinks=4, dtype=1,
             scale=0.125, flags=0)
    d.update(kw)
    return gdn.SwaDesc(**d)


BAD = [(dict(dtype=3), 3), (dict(dtype=-1), 3), (dict(batch=0), 2), (dict(seqlen=-1), 2), (dict(keylen=-1), 2),
       (dict(num_seqs=0), 2), (dict(window=0), 2), (dict(sinks=-1), 2), (dict(heads=0), 2), (dict(kv_heads=0), 2),
       (dict(heads=7), 2), (dict(heads=34, kv_heads=2), 5), (dict(heads=1040, kv_heads=65), 5), (dict(dim=96), 5),
       (dict(dim=512), 5), (dict(dim=256, dtype=0), 5), (dict(sinks=129), 5), (dict(scale=0.0), 5),
       (dict(scale=-1.0), 5), (dict(scale=float("inf")), 5), (dict(scale=float("nan")), 5), (dict(flags=1), 5),
       (dict(batch=1, num_seqs=1 << 30, heads=64, kv_heads=64), 2), (dict(batch=1 << 15, seqlen=1 << 15), 2), (dict(batch=1 << 15, keylen=1 << 15), 2)]


@pytest.mark.parametrize("kw,code", BAD)
def test_descriptor(lib, kw, code):
    n = ctypes.c_size_t(0)
    for size in (lib.gdn_swa_fwd_workspace_size, lib.gdn_swa_bwd_workspace_size):
        assert size(desc(**kw), ctypes.byref(n)) == code
        assert lib.gdn_last_error_message()


def test_workspace(lib):
    n = ctypes.c_size_t(0)
    for size in (lib.gdn_swa_fwd_workspace_size, lib.gdn_swa_bwd_workspace_size):
        assert size(desc(), ctypes.byref(n)) == 0 and n.value >= 256
        assert size(desc(), None) == 1 and size(None, ctypes.byref(n)) == 1
    assert lib.gdn_swa_bwd_workspace_size(desc(dim=256), ctypes.byref(n)) == 5       # forward only
    assert lib.gdn_swa_fwd_workspace_size(desc(dim=256), ctypes.byref(n)) == 0
    assert gdn.swa_fwd_workspace_size(1, 50408, 50408, 16, 16, 128, 8, 2048) > 256
    assert gdn.swa_bwd_workspace_size(1, 32768, 32768, 16, 8, 64, 1, 2048, 16) > 16 * 32768 * 4
    with pytest.raises(gdn.GdnError, match="GDN_ERR_UNSUPPORTED"):
        gdn.swa_bwd_workspace_size(1, 8, 8, 1, 1, 256, 1, 4)


def test_fwd_refusals(lib):
    def call(d=None, q=A, k=B, v=C, cu=None, cuk=None, o=D_, lse=E, ws=WS, size=BIG):
        return lib.gdn_swa_fwd(d or desc(), q, k, v, cu, cuk, o, lse, ws, size, None)

    assert call(d=desc(window=0)) == 2
    for name in "qkvo":
        assert call(**{name: None}) == 1 and call(**{name: F + 8}) == 4, name
    assert call(lse=E + 2) == 4
    assert call(cu=F) == 1 and call(cuk=F) == 1                          # one without the other
    assert call(cu=F, cuk=G) == 2                                        # packed with batch 2
    one = desc(batch=1, num_seqs=3)
    assert call(d=one, cu=F, cuk=G, ws=None) == 6 and call(d=one, cu=F, cuk=G, size=8) == 6
    assert call(d=one, cu=F, cuk=G, ws=WS + 4) == 4 and call(d=one, cu=F, cuk=G, ws=A) == 8
    assert call(d=one, cu=F + 2, cuk=G) == 4 and call(d=one, cu=F, cuk=G + 1) == 4
    assert call(d=desc(num_seqs=3)) == 2
    assert call(o=A) == 8 and call(o=B + 64) == 8 and call(lse=D_ + 16) == 8 and call(lse=C) == 8
    assert b"overlaps" in lib.gdn_last_error_message()


def test_bwd_refusals(lib):
    def call(d=None, g=A, q=B, k=C, v=D_, o=E, lse=F, cu=None, cuk=None, dq=G, dk=H, dv=I, ws=WS, size=BIG):
        return lib.gdn_swa_bwd(d or desc(), g, q, k, v, o, lse, cu, cuk, dq, dk, dv, ws, size, None)

    for name in ("g", "q", "k", "v", "o", "dq", "dk", "dv"):
        assert call(**{name: None}) == 1 and call(**{name: J + 8}) == 4, name
    assert call(lse=None) == 1 and call(lse=F + 2) == 4 and call(ws=None) == 6 and call(size=256) == 6
    assert call(cu=J) == 1 and call(cu=J, cuk=K) == 2 and call(d=desc(dim=256)) == 5
    assert call(dq=A) == 8 and call(dk=C) == 8 and call(dv=H + 16) == 8 and call(dq=F) == 8 and call(ws=I) == 8


def cache(**kw):
    d = dict(slots=8, kv_heads=2, window=32, sinks=4, dim=64, dtype=1)
    d.update(kw)
    return gdn.CacheDesc(**d)


CACHE_BAD = [(dict(slots=0), 2), (dict(kv_heads=0), 2), (dict(window=0), 2), (dict(sinks=-1), 2), (dict(dtype=4), 3),
             (dict(dtype=-1), 3), (dict(slots=65537), 5), (dict(kv_heads=1025), 5), (dict(dim=48), 5),
             (dict(sinks=129), 5), (dict(window=1 << 28), 5)]


@pytest.mark.parametrize("kw,code", CACHE_BAD)
def test_cache_descriptor(lib, kw, code):
    n = ctypes.c_size_t(0)
    assert lib.gdn_swa_step_workspace_size(cache(**kw), 4, 8, ctypes.byref(n)) == code
    assert lib.gdn_cache_write(cache(**kw), 4, 40, 1, A, B, None, None, None, C, None, None, None) == code
    assert lib.gdn_cache_read(cache(**kw), 4, 40, 1, C, None, D_, None, None, A, B, None, None) == code


@pytest.mark.parametrize("read", [False, True])
def test_cache_refusals(lib, read):
    def call(d=None, N=4, T=40, dt=1, k=A, v=B, cu=None, lengths=C, slots=None, cache_=D_, scales=None, status=None):
        d = d or cache()
        if read:
            return lib.gdn_cache_read(d, N, T, dt, cache_, scales, lengths, slots, cu, k, v, status, None)
        return lib.gdn_cache_write(d, N, T, dt, k, v, cu, lengths, slots, cache_, scales, status, None)

    assert call(N=-1) == 2 and call(N=4097, d=cache(slots=5000)) == 5 and call(T=-1) == 2 and call(T=41) == 2
    assert call(T=1 << 30) == 2 and call(N=0, T=4) == 2
    assert call(N=9, T=45) == 2 and b"slots" in lib.gdn_last_error_message()      # more sequences than slots
    assert call(dt=3) == 3 and call(dt=0) == 5 and call(dt=2) == 5
    assert call(scales=E) == 5 and call(d=cache(dtype=3)) == 1                    # scales with 8 bits alone
    assert call(k=None) == 1 and call(v=None) == 1 and call(cache_=None) == 1
    if read:
        assert call(lengths=None) == 1
    assert call(k=A + 8) == 4 and call(cache_=D_ + 8) == 4 and call(lengths=C + 2) == 4 and call(slots=E + 2) == 4
    assert call(status=E + 1) == 4 and call(cu=E + 2) == 4 and call(d=cache(dtype=3), scales=E + 2) == 4
    assert call(k=D_) == 8 and call(status=D_) == 8 and call(status=C) == 8
    if read:
        assert call(k=B + 16) == 8
    assert call(N=0, T=0, k=None, v=None, cache_=None, lengths=None) == 0


def test_step_refusals(lib):
    def call(d=None, N=4, h=8, dt=1, scale=0.1, q=A, k=B, v=C, lengths=D_, slots=None, cache_=E, scales=None, o=F,
             ws=WS, size=BIG, status=None):
        return lib.gdn_swa_step(d or cache(), N, h, dt, scale, q, k, v, lengths, slots, cache_, scales, o, ws, size,
                                status, None)

    assert call(N=-1) == 2 and call(N=4097, d=cache(slots=5000)) == 5 and call(N=9) == 2
    assert call(h=7) == 2 and call(h=64) == 5 and call(dt=3) == 3 and call(dt=0) == 5
    assert call(d=cache(dtype=0, dim=256), dt=0) == 5
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=scale) == 5
    assert call(scales=G) == 5 and call(d=cache(dtype=3)) == 1
    for name in ("q", "k", "v", "lengths", "cache_", "o"):
        assert call(**{name: None}) == 1, name
    assert call(q=A + 8) == 4 and call(o=F + 4) == 4 and call(lengths=D_ + 1) == 4 and call(status=G + 2) == 4
    wide = cache(window=4096)
    assert call(d=wide, ws=None) == 6 and call(d=wide, size=16) == 6
    assert call(o=A) == 8 and call(o=E + 64) == 8 and call(q=E) == 8 and call(status=D_) == 8 and call(d=wide, ws=F) == 8
    assert call(N=0, q=None, k=None, v=None, lengths=None, cache_=None, o=None) == 0
    n = ctypes.c_size_t(0)
    assert lib.gdn_swa_step_workspace_size(cache(), 4, 8, None) == 1
    assert lib.gdn_swa_step_workspace_size(None, 4, 8, ctypes.byref(n)) == 1
    assert lib.gdn_swa_step_workspace_size(cache(), 4, 9, ctypes.byref(n)) == 2


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 2, 32)
    c = torch.zeros(2, 3, 2, 8, 32)
    n = torch.zeros(1, dtype=torch.int32)
    for f in (lambda: gdn.swa_fwd(x, x, x, 4), lambda: gdn.swa_bwd(x, x, x, x, x, x[..., 0], 4),
              lambda: gdn.swa_step(c, x[0], x[0], x[0], n), lambda: gdn.cache_write(c, x, x),
              lambda: gdn.cache_read(c, n)):
        with pytest.raises(ValueError, match="expected a GPU"):
            f()
    with pytest.raises(TypeError):
        gdn.swa_fwd([1.0], x, x, 4)


def test_header_names_every_call():
    """The header's declarations and the binding's agree on what there is."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(gdn.HERE), "include", "gdn.h")).read()
    declared = set(re.findall(r"gdn_status (gdn_\w+)\(", text))
    lib = gdn.load()
    assert {"gdn_swa_fwd", "gdn_swa_bwd", "gdn_swa_step", "gdn_cache_write", "gdn_cache_read"} <= declared
    assert all(hasattr(lib, name) for name in declared)
