"""The fp64 oracle of the gated linear recurrence, layer norm and the state
moves, pinned to closed forms and to central finite differences (CPU)."""
import numpy as np

from oracle import operators as R

CU = [0, 3, 3, 4, 9]      # a packed batch with an empty and a one-token sequence


def _scan_inputs(seed=0, T=9, D=3):
    g = np.random.default_rng(seed)
    return (g.standard_normal((1, T, D)), -g.uniform(0.01, 1.0, (1, T, D)), g.standard_normal((4, D)),
            g.standard_normal((1, T, D)), g.standard_normal((4, D)))


def test_scan_closed_forms():
    x, la, init, _, _ = _scan_inputs()
    h, fin = R.scan(x, np.zeros_like(la), init, CU)                 # no decay: sums
    assert np.allclose(h[0, 3:4], init[2] + x[0, 3:4]) and np.allclose(h[0, 8], init[3] + x[0, 4:].sum(0))
    assert np.allclose(fin, [h[0, 2], init[1], h[0, 3], h[0, 8]])   # the empty sequence keeps its state
    h, _ = R.scan(x, np.full_like(la, -np.inf), init, CU)           # everything is forgotten
    assert np.array_equal(h, x)
    h, fin = R.scan(np.zeros_like(x), la, init, CU)                 # pure decay
    assert np.allclose(fin[3], init[3] * np.exp(la[0, 4:].sum(0)))


def test_scan_gradients_by_differences():
    x, la, init, gh, gf = _scan_inputs(1)

    def loss(x, la, init):
        h, fin = R.scan(x, la, init, CU)
        return (gh * h).sum() + (gf * fin).sum()

    grads = R.scan_bwd(la, R.scan(x, la, init, CU)[0], gh, init, gf, CU)
    for i, (v, got) in enumerate(zip((x, la, init), grads)):
        for at in np.ndindex(v.shape):
            args = [[x, la, init], [x, la, init]]
            for k, s in enumerate((1e-6, -1e-6)):
                args[k][i] = v.copy()
                args[k][i][at] += s
            assert abs((loss(*args[0]) - loss(*args[1])) / 2e-6 - got[at]) < 1e-7


def test_layernorm_rows_and_gradients():
    g = np.random.default_rng(2)
    x, dy, w, b = g.standard_normal((4, 5)) + 3, g.standard_normal((4, 5)), g.standard_normal(5), g.standard_normal(5)
    y, mean, rstd = R.layernorm(x, eps=0.0)
    assert np.allclose(y.mean(1), 0) and np.allclose((y * y).mean(1), 1)
    assert np.allclose(R.layernorm(x, w, b, 0.0)[0], y * w + b)
    _, mean, rstd = R.layernorm(x, eps=1e-2)
    grads = R.layernorm_bwd(dy, x, mean, rstd, w)
    loss = lambda x, w, b: (dy * R.layernorm(x, w, b, 1e-2)[0]).sum()   # noqa: E731
    for i, (v, got) in enumerate(zip((x, w, b), grads)):
        for at in np.ndindex(v.shape):
            lo, hi = [x, w, b], [x, w, b]
            lo[i], hi[i] = v.copy(), v.copy()
            lo[i][at] -= 1e-6
            hi[i][at] += 1e-6
            assert abs((loss(*hi) - loss(*lo)) / 2e-6 - got[at]) < 1e-7


def test_state_move():
    s = np.arange(8.0).reshape(1, 4, 2)
    assert np.array_equal(R.state_move(s, [1, 0, -1], [0, 1, 3])[0], [[2, 3], [0, 1], [4, 5], [0, 0]])
