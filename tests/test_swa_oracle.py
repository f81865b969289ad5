"""The oracle of windowed attention pinned to closed forms, to central differences and to the cache's own rules."""
import numpy as np
import pytest

from oracle import attention as A


def draw(seed, *shapes):
    g = np.random.default_rng(seed)
    return [g.standard_normal(s) for s in shapes]


def test_window_of_one_is_the_value_itself():
    q, k, v = draw(0, (1, 5, 2, 4), (1, 5, 2, 4), (1, 5, 2, 4))
    o, lse = A.attention(q, k, v, 1)
    assert np.allclose(o, v) and np.allclose(lse, (q * k).sum(-1) / 2)


def test_equal_keys_give_the_mean_of_what_is_seen():
    _, _, v = draw(1, (1,), (1,), (1, 9, 1, 3))
    q, k = np.ones((1, 9, 1, 3)), np.ones((1, 9, 1, 3))
    o, lse = A.attention(q, k, v, 3, 2)
    for i in range(9):
        see = [j for j in range(i + 1) if i - j < 3 or j < 2]
        assert np.allclose(o[0, i, 0], v[0, see, 0].mean(0))
        assert np.isclose(lse[0, i, 0], np.sqrt(3) + np.log(len(see)))


def test_wide_window_is_causal_softmax():
    q, k, v = draw(2, (2, 7, 2, 4), (2, 7, 1, 4), (2, 7, 1, 4))
    o, _ = A.attention(q, k, v, 100)
    s = np.einsum("bihd,bjd->bhij", q, k[:, :, 0]) / 2
    s[:, :, np.triu_indices(7, 1)[0], np.triu_indices(7, 1)[1]] = -np.inf
    p = np.exp(s - s.max(-1, keepdims=True))
    want = np.einsum("bhij,bjd->bihd", p / p.sum(-1, keepdims=True), v[:, :, 0])
    assert np.allclose(o, want)


def test_sequences_and_positions():
    """Packed is separate; queries behind keys are the last rows of the whole; those before every key see nothing."""
    q, k, v = draw(3, (1, 12, 2, 4), (1, 12, 1, 4), (1, 12, 1, 4))
    o, lse = A.attention(q, k, v, 4, 1, [0, 5, 5, 12])
    for a, b in ((0, 5), (5, 12)):
        po, pl = A.attention(q[:, a:b], k[:, a:b], v[:, a:b], 4, 1)
        assert np.array_equal(o[:, a:b], po) and np.array_equal(lse[:, a:b], pl)
    whole, _ = A.attention(q, k, v, 4, 1)
    last, _ = A.attention(q[:, 9:], k, v, 4, 1)
    assert np.allclose(last, whole[:, 9:])
    o, lse = A.attention(q, k[:, :4], v[:, :4], 4)
    assert not o[:, :8].any() and (lse[:, :8] == -np.inf).all() and np.isfinite(lse[:, 8:]).all()


@pytest.mark.parametrize("T,Tk,window,sinks,cu,cuk", [(6, 6, 3, 1, None, None), (4, 7, 3, 2, None, None),
                                                      (6, 4, 3, 1, None, None), (6, 6, 2, 1, [0, 2, 6], [0, 3, 6])])
def test_gradients_are_differences(T, Tk, window, sinks, cu, cuk):
    q, k, v, w = draw(4, (1, T, 2, 3), (1, Tk, 1, 3), (1, Tk, 1, 3), (1, T, 2, 3))
    o, lse = A.attention(q, k, v, window, sinks, cu, cuk, 0.7)
    got = A.attention_bwd(w, q, k, v, o, lse, window, sinks, cu, cuk, 0.7)
    for x, g in zip((q, k, v), got):
        flat = x.reshape(-1)
        for at in range(flat.size):
            keep, side = flat[at], []
            for h in (1e-6, -1e-6):
                flat[at] = keep + h
                side.append((A.attention(q, k, v, window, sinks, cu, cuk, 0.7)[0] * w).sum())
            flat[at] = keep
            assert abs(g.reshape(-1)[at] - (side[0] - side[1]) / 2e-6) < 1e-8


def test_cache_rows():
    assert [A.cache_row(p, 3, 2) for p in range(9)] == [0, 1, 2, 3, 4, 2, 3, 4, 2]
    for length in range(12):          # what is read back are the sinks and the last `window`, in order
        k = np.arange(length, dtype=float).reshape(1, length, 1, 1)
        cache, _ = A.cache_write(np.full((2, 1, 1, 5, 1), -1.0), k, -k, [0], 2)
        (rk, rv), = A.cache_read(cache, [length], 2)
        want = [p for p in range(length) if p < 2 or p >= length - 3]
        assert rk[:, 0, 0].tolist() == want and np.array_equal(rv, -rk)


def test_step_is_the_last_row_of_the_whole():
    k, v, q = draw(6, (1, 20, 2, 4), (1, 20, 2, 4), (1, 4, 4))
    cache, _ = A.cache_write(np.zeros((2, 1, 2, 7, 4)), k[:, :19], v[:, :19], [0], 2)
    o, _, _ = A.step(cache, q, k[:, 19], v[:, 19], [19], 2)
    want, _ = A.attention(q[:, None], k, v, 5, 2)
    assert np.allclose(o, want[:, 0])
    o, same, _ = A.step(cache, q, k[:, 19], v[:, 19], [19], 2, slots=[-1])
    assert not o.any() and np.array_equal(same, cache)


def test_e4m3():
    assert A.e4m3([448.0, -1.0])[1] == 1 and A.e4m3([448.1, 1.0])[1] == 2 and A.e4m3([3.5, 0.0])[1] == 2.0 ** -7
    y, s = A.e4m3([1.75, 0.1, -0.3, 0.0])
    assert s == 2.0 ** -8 and y.tolist() == [448.0, 26.0, -80.0, 0.0]
    assert A.e4m3([0.0])[1] == 2.0 ** -126 and np.isnan(A.e4m3([1.0, np.inf])[0]).all()
    x = np.random.default_rng(0).standard_normal(1000)
    y, s = A.e4m3(x)
    assert (np.abs(y * s - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s)).all()
    y, _ = A.e4m3([448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])       # halves to even, subnormals too
    assert y.tolist() == [448.0, 16.0, 20.0, 0.0, 2 * 2.0 ** -9]
