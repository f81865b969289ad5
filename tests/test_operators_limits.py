"""Layer norm and state moves where a block takes several turns, a call several
launches or a tensor more than 2^31 values."""
import pytest
import torch

import gated_delta_rule_24_amd as gdn

from .op_util import DT
from .test_layernorm import check_bwd, check_fwd, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [1500, 1600, 2048, 2049, 4100, 6144, 8192, 8200, 8201, 12290, 16384])
def test_layernorm_forward_in_turns(D):
    """Rows over one wave and over several, more of them than the 8192 blocks take at once: the last turn's rows
    have the bits of a call of their own, which is within its bounds."""
    rows = 8192 * (4 if D <= 1536 else 2 if D <= 2048 else 1) + 70     # a block holds 4, 2 or 1 rows at a time
    x, w, b, _ = make(40, D, ("bf16", "bf16"), seed=D)
    big = torch.empty(rows, D, dtype=DT["bf16"], device="cuda").normal_()
    big[-40:] = x
    part = check_fwd(40, D, ("bf16", "bf16"), seed=D)[3:]
    for got, want in zip(gdn.layernorm_fwd(big, w, b, out_dtype=DT["bf16"]), part):
        assert torch.equal(got[-40:], want)


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("D", [1032, 2048, 2050, 4096, 4100, 8192, 8201, 16384])
def test_layernorm_gradient_in_turns(D, types):
    """1030 rows of one to sixteen waves: blocks of every layout take at least two of them, one after the other."""
    check_bwd(1030 if D < 8000 else 530, D, types, seed=D)


def test_layernorm_sums_over_many_rows_are_exact():
    """Over 2^31 values: sums of small whole numbers below 2^24 have no rounding, so a row that is lost or counted
    twice shows in dweight and in dbias."""
    rows, D = 2_200_000, 1000
    r = torch.arange(rows, device="cuda")
    dy = ((r * 7 + r // 512) % 3).to(torch.bfloat16)[:, None].expand(rows, D).contiguous()
    x = (1 + (r * 5 + r // 2048) % 2).to(torch.bfloat16)[:, None].expand(rows, D).contiguous()
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    _, dw, db = gdn.layernorm_bwd(dy, x, mean, rstd)
    want_w, want_b = int((dy[:, 0].long() * x[:, 0].long()).sum()), int(dy[:, 0].long().sum())
    assert 2 ** 20 < want_b < want_w < 2 ** 24
    assert (dw == want_w).all() and (db == want_b).all()


def test_more_layers_than_one_launch():
    """Over 65535 layers: two launches, one after the other, over chains (pages that are read and written) and forks."""
    L = 70_000
    state = torch.arange(L * 3 * 2, dtype=torch.int32, device="cuda").view(L, 3, 2)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")     # noqa: E731
    status = i32(-7, -7)
    for src, dst in (((1, 0, 2), (0, 1, 2)), ((2, 2), (0, 1)), ((-1,), (2,))):
        want = state.clone()
        for a, b in zip(src, dst):
            want[:, b] = state[:, a] if a >= 0 else 0
        gdn.state_move(state, i32(*src), i32(*dst), layers=True, status=status)
        assert torch.equal(state, want) and gdn.state_move_check(status) == 0
