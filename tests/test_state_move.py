"""Moves of resident states: bytes are copied, so every check is for equality."""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn
from oracle import operators as R

from .op_util import host

pytestmark = pytest.mark.gpu


def idx(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


def check(shape, src, dst, dtype=torch.float32, layers=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = torch.randn(shape, generator=g, device="cuda").to(dtype)
    full = state if layers else state[None]
    want = R.state_move(host(full), src, dst)
    status = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    got = gdn.state_move(state, idx(src), idx(dst), layers=layers, status=status)
    assert got is state
    assert np.array_equal(host(full), want)
    assert gdn.state_move_check(status) == 0 and status.tolist() == [len(src), 0]


@pytest.mark.parametrize("page", [(1,), (3,), (4,), (33,), (16, 16), (2, 31, 17), (4, 128, 128)], ids=str)
@pytest.mark.parametrize("layers", [1, 3])
def test_patterns(page, layers):
    P = 12
    shape = (layers, P) + page
    check(shape, [5] * 7, [0, 1, 2, 3, 4, 6, 11])               # fork
    check(shape, [11, 10, 9], [0, 4, 7])                        # compact
    check(shape, [-1, -1], [3, 8])                              # free
    check(shape, list(range(1, P)), list(range(P - 1)))         # a chain down
    check(shape, list(range(P - 1)), list(range(1, P)))         # a chain up
    check(shape, [1, 2, 3, 0, 7, 6], [0, 1, 2, 3, 6, 7])        # cycles
    check(shape, [4, 4, -1, 4], [4, 5, 6, 0])                   # onto itself, with copies and a freed slot
    check(shape, [], [])


@pytest.mark.parametrize("moves", [1, 2, 3, 15, 16, 17, 255, 256, 257, 1000, 1024, 1025, 2049, 4096])
def test_counts(moves):
    g = np.random.default_rng(moves)
    P = moves + 5
    for page in ((96,), (7,), (1030,)):
        check((2, P) + page, g.integers(-1, P, moves), g.permutation(P)[:moves])
    check((P, 40), np.roll(np.arange(moves), 1), np.arange(moves), layers=False)


def test_types_and_one_layer():
    check((6, 8, 4), [0, 1], [1, 0], torch.bfloat16, layers=False)
    check((6, 10), [0, 1], [1, 0], torch.float64, layers=False)
    check((5, 3, 6), [2], [0], torch.int32)
    s = torch.zeros(5, 4, 3, dtype=torch.bfloat16, device="cuda")
    gdn.state_move(s, idx([1]), idx([0]))                        # 24 bytes a page
    with pytest.raises(gdn.GdnError, match="multiple of 4"):
        gdn.state_move(torch.zeros(5, 3, dtype=torch.bfloat16, device="cuda"), idx([1]), idx([0]))


@pytest.mark.parametrize("src,dst,code", [([6], [0], 1), ([-2], [0], 1), ([0], [-1], 2), ([0], [6], 2),
                                          ([0, 1], [2, 2], 3), ([2 ** 31 - 1], [0], 1), ([0], [-2 ** 31], 2),
                                          ([0] * 5 + [9], [5, 4, 3, 2, 1, 0], 1)])
def test_bad_indices_change_nothing(src, dst, code):
    state = torch.randn(3, 6, 1000, device="cuda")
    keep, status = state.clone(), torch.empty(2, dtype=torch.int32, device="cuda")
    gdn.state_move(state, idx(src), idx(dst), layers=True, status=status)
    assert gdn.state_move_check(status) == code
    gdn.state_move(state, idx(src), idx(dst), layers=True)
    assert torch.equal(state, keep)


def test_infinite_and_nan_bytes():
    state = torch.tensor([float("nan"), float("inf"), -0.0, 1.0], device="cuda").view(4, 1)
    bits = state.view(torch.int32).clone()
    gdn.state_move(state, idx([0, 1, 2]), idx([1, 2, 3]))
    assert torch.equal(state.view(torch.int32), bits[[0, 0, 1, 2]])


def test_graph_replays_and_streams():
    state = torch.randn(2, 9, 5000, device="cuda")
    src, dst, ref = idx(np.roll(np.arange(9), 1)), idx(np.arange(9)), None
    ref = state.clone()
    graph = torch.cuda.CUDAGraph()
    gdn.state_move(state, src, dst, layers=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gdn.state_move(state, src, dst, layers=True)
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(state, ref.roll(k + 2, 1))
    a, b = torch.randn(64, 30000, device="cuda"), torch.randn(64, 30000, device="cuda")
    wa, wb = a.roll(1, 0), b.roll(-1, 0)
    s, d = idx(np.roll(np.arange(64), 1)), idx(np.arange(64))
    t = idx(np.roll(np.arange(64), -1))
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        gdn.state_move(a, s, d)
    with torch.cuda.stream(torch.cuda.Stream()):
        gdn.state_move(b, t, d)
    torch.cuda.synchronize()
    assert torch.equal(a, wa) and torch.equal(b, wb)


def test_offsets_past_32_bits():
    state = torch.zeros(2, 5, 1 << 29, dtype=torch.float32, device="cuda")     # 2 GiB a page
    state[1, 4, -3:] = 5.0
    gdn.state_move(state, idx([4]), idx([3]), layers=True)
    assert state[1, 3, -3:].tolist() == [5.0] * 3 and not state[1, 3, :-3].any()


def test_refusals():
    s = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError, match="dims"):
        gdn.state_move(s, idx([0]), idx([1]), layers=True)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.state_move(s.t(), idx([0]), idx([1]))
    with pytest.raises(ValueError, match="dtype"):
        gdn.state_move(s, idx([0]).long(), idx([1]))
    with pytest.raises(ValueError, match="must be"):
        gdn.state_move(s, idx([0]), idx([1, 2]))
    with pytest.raises(gdn.GdnError, match="moves"):
        gdn.state_move(s, idx([0] * 5), idx(range(5)))
