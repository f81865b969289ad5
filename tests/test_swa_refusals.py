"""Calls of windowed attention that end in the library's own refusal, or in a result, where they are odd."""
import ctypes

import pytest
import torch

import gated_delta_rule_24_amd as gdn


def test_scales_past_the_largest():
    """scale log2(e) has to be finite: 0 times it is a score."""
    lib, n = gdn.load(), ctypes.c_size_t(0)
    p = 0x100000000
    for scale, code in ((2.0 ** 127, 0), (2.4e38, 5), (3.4e38, 5), (1e-45, 0)):
        desc = gdn.SwaDesc(1, 4, 4, 1, 1, 32, 1, 4, 0, 1, scale, 0)
        assert lib.gdn_swa_fwd_workspace_size(desc, ctypes.byref(n)) == code
        assert lib.gdn_swa_bwd_workspace_size(desc, ctypes.byref(n)) == code
        cache = gdn.CacheDesc(1, 1, 4, 0, 32, 1)
        if code:
            assert lib.gdn_swa_step(cache, 1, 1, 1, scale, p, 2 * p, 3 * p, 4 * p, None, 5 * p, None, 6 * p, None, 0, None,
                                    None) == code


@pytest.mark.gpu
def test_heads_of_no_elements():
    q = torch.empty(1, 4, 2, 0, device="cuda")
    c = torch.empty(2, 3, 2, 8, 0, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in (lambda: gdn.swa_fwd(q, q, q, 4), lambda: gdn.swa_bwd(q, q, q, q, q, torch.empty(1, 4, 2, device="cuda"), 4),
                 lambda: gdn.swa_step(c, q[:, 0], q[:, 0], q[:, 0], n)):
        with pytest.raises(gdn.GdnError, match="GDN_ERR_UNSUPPORTED"):
            call()
