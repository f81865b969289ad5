"""Calls of windowed attention that end in the library's own refusal, or in a result, where they are odd."""
import ctypes

import pytest
import torch

import gated_delta_rule_24_amd as gdn


@pytest.mark.gpu
def test_heads_of_no_elements():
    q = torch.empty(1, 4, 2, 0, device="cuda")
    c = torch.empty(2, 3, 2, 8, 0, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in (lambda: gdn.swa_fwd(q, q, q, 4), lambda: gdn.swa_bwd(q, q, q, q, q, torch.empty(1, 4, 2, device="cuda"), 4),
                 lambda: gdn.swa_step(c, q[:, 0], q[:, 0], q[:, 0], n)):
        with pytest.raises(gdn.GdnError, match="GDN_ERR_UNSUPPORTED"):
            call()
