"""The operators as they are used together: a recurrent block trained, a batch of
resident sequences served."""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn
import workloads as W
from oracle import operators as R

from .gpu_util import check_parity, run_chunk
from .op_util import dev, host

pytestmark = pytest.mark.gpu


def test_block_forward_and_backward():
    """norm -> recurrence -> norm over a packed batch in fp32, forward and gradients, against the fp64 chain.
    Each stage is within its own tests' bounds; joined, 1e-4 of the result's size leaves two digits of room."""
    g = np.random.default_rng(0)
    T, D, cu = 600, 72, [0, 200, 200, 201, 600]
    x, la = g.standard_normal((T, D)), -g.uniform(0.01, 0.3, (1, T, D))
    w1, b1, w2, b2 = (g.standard_normal(D) for _ in range(4))
    init, dy = g.standard_normal((4, D)), g.standard_normal((T, D))
    t = [dev(v) for v in (x, la, w1, b1, w2, b2, init, dy)]
    x, la, w1, b1, w2, b2, init, dy = (host(v) for v in t)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")

    y1, m1, r1 = gdn.layernorm_fwd(t[0], t[2], t[3])
    h, fin = gdn.scan_fwd(y1[None], t[1], t[6], cut)
    y2, m2, r2 = gdn.layernorm_fwd(h[0], t[4], t[5])
    dh, dw2, db2 = gdn.layernorm_bwd(t[7], h[0], m2, r2, t[4])
    dy1, dla, dinit = gdn.scan_bwd(t[1], h, dh[None], t[6], None, cut)
    dx, dw1, db1 = gdn.layernorm_bwd(dy1[0], t[0], m1, r1, t[2])

    ry1, rm1, rr1 = R.layernorm(x, w1, b1)
    rh, rfin = R.scan(ry1[None], la, init, cu)
    ry2, rm2, rr2 = R.layernorm(rh[0], w2, b2)
    rdh, rdw2, rdb2 = R.layernorm_bwd(dy, rh[0], rm2, rr2, w2)
    rdy1, rdla, rdinit = R.scan_bwd(la, rh, rdh[None], init, None, cu)
    rdx, rdw1, rdb1 = R.layernorm_bwd(rdy1[0], x, rm1, rr1, w1)
    for got, want in ((y2, ry2), (fin, rfin), (dx, rdx), (dla, rdla), (dinit, rdinit), (dw1, rdw1), (db1, rdb1),
                      (dw2, rdw2), (db2, rdb2)):
        assert np.abs(host(got) - want).max() <= 1e-4 * np.sqrt((want ** 2).mean())


def test_head_norm_behind_the_delta_rule():
    """chunk_fwd's output normed per head: the norm of the fp64 norm's input is the kernel's own o."""
    inp = W.chunk_inputs(2, 130, 3, 64, 48, "bf16", seed=91, name="norm behind chunk_fwd")
    o, S = run_chunk(inp)
    check_parity(inp, o, S)
    y, mean, rstd = gdn.layernorm_fwd(o, out_dtype=torch.bfloat16)
    want = R.layernorm(host(o).reshape(-1, 48))[0].reshape(o.shape)
    assert y.shape == o.shape and np.abs(host(y) - want).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-5


def test_serving_with_forks_and_compaction():
    """Resident states of both rules: prefill, fork one prompt, step, end sequences, compact, step on.  Every
    sequence gets the bits that it gets in a batch where nothing is moved."""
    H, dk, dv, N, D = 2, 64, 32, 6, 48
    g = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")        # noqa: E731
    pool, chan = torch.zeros(N, H, dv, dk, device="cuda"), torch.zeros(N, D, device="cuda")
    q, k, v = (torch.nn.functional.normalize(new(1, 20, H, d), dim=-1) for d in (dk, dk, dv))
    la, beta = -0.1 * torch.rand(1, 20, H, generator=g, device="cuda"), torch.rand(1, 20, H, generator=g,
                                                                                   device="cuda")
    gdn.chunk_fwd(q, k, v, la, beta, final_state=pool[2:3])
    gdn.scan_fwd(new(1, 20, D), -new(1, 20, D).abs(), final_state=chan[2:3])
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for s in (pool, chan):
        gdn.state_move(s, i32(2, 2, 2), i32(0, 1, 3))                   # four samples of one prompt
    assert all(torch.equal(pool[j], pool[2]) and torch.equal(chan[j], chan[2]) for j in (0, 1, 3))

    def step(pool, chan, who, t):
        gg = torch.Generator(device="cuda").manual_seed(100 + t)
        draw = lambda *s: torch.randn(4, *s, generator=gg, device="cuda")[who].contiguous()   # noqa: E731
        o = gdn.decode_step(pool, draw(H, dk) / 8, draw(H, dk) / 8, draw(H, dv), -draw(H).abs(), draw(H).sigmoid())
        return o, gdn.scan_step(chan, draw(D), -draw(D).abs())

    still = pool[:4].clone(), chan[:4].clone()
    moved = pool[:4].clone(), chan[:4].clone()
    a, b = step(*still, [0, 1, 2, 3], 0), step(*moved, [0, 1, 2, 3], 0)
    assert all(torch.equal(p, r) for p, r in zip(a, b))
    for s in moved:                     # sequences 0 and 1 end; 3 and 2 move into their slots
        gdn.state_move(s, i32(3, 2, -1, -1), i32(0, 1, 2, 3))
        assert not s[2:].any()
    moved = tuple(s[:2] for s in moved)
    for t in range(1, 4):
        a, b = step(*still, [0, 1, 2, 3], t), step(*moved, [3, 2], t)
        assert all(torch.equal(p[[3, 2]], r) for p, r in zip(a, b))
        assert all(torch.equal(p[[3, 2]], r) for p, r in zip(still, moved))
