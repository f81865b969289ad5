"""Windowed attention and its cache as they are used: a hybrid block trained, resident sequences prefilled, stepped,
forked, compacted and continued."""
import numpy as np
import pytest
import torch

import gated_delta_rule_24_amd as gdn
from oracle import attention as A
from oracle import operators as R

from .op_util import HALF, cu_tensor, dev, host

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def draw(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def test_block_forward_and_backward():
    """norm -> attention -> norm over a packed batch in fp32, forward and gradients, against the fp64 chain.  Each
    stage is within its own tests' bounds; joined, 1e-4 of the result's size leaves two digits of room."""
    g = np.random.default_rng(0)
    T, H, d, cu, window, sinks = 90, 2, 32, [0, 30, 30, 31, 90], 12, 2
    x, w1, b1, w2, b2 = (dev(g.standard_normal(s)) for s in ((T, H * d), H * d, H * d, d, d))
    dy = dev(g.standard_normal((T, H, d)))
    c = cu_tensor(cu)
    y1, m1, r1 = gdn.layernorm_fwd(x, w1, b1)
    qkv = y1.view(1, T, H, d)
    o, lse = gdn.swa_fwd(qkv, qkv, qkv, window, sinks, c)
    y2, m2, r2 = gdn.layernorm_fwd(o, w2, b2)
    do, dw2, db2 = gdn.layernorm_bwd(dy[None], o, m2, r2, w2)
    grads = gdn.swa_bwd(do, qkv, qkv, qkv, o, lse, window, sinks, c)
    dx, dw1, db1 = gdn.layernorm_bwd(sum(grads).view(T, H * d), x, m1, r1, w1)

    hx, hw1, hb1, hw2, hb2, hdy = (host(v) for v in (x, w1, b1, w2, b2, dy))
    ry1, rm1, rr1 = R.layernorm(hx, hw1, hb1)
    rq = ry1.reshape(1, T, H, d)
    ro, rl = A.attention(rq, rq, rq, window, sinks, cu)
    ry2, rm2, rr2 = R.layernorm(ro.reshape(-1, d), hw2, hb2)
    rdo, rdw2, rdb2 = R.layernorm_bwd(hdy.reshape(-1, d), ro.reshape(-1, d), rm2, rr2, hw2)
    rg = A.attention_bwd(rdo.reshape(rq.shape), rq, rq, rq, ro, rl, window, sinks, cu)
    rdx, rdw1, rdb1 = R.layernorm_bwd(sum(rg).reshape(T, H * d), hx, rm1, rr1, hw1)
    for got, want in ((y2, ry2), (dx, rdx), (dw1, rdw1), (db1, rdb1), (dw2, rdw2), (db2, rdb2)):
        worst = np.abs(host(got).reshape(want.shape) - want).max() / np.sqrt((want ** 2).mean())
        assert worst <= 1e-4


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_serving(kind):
    """Prompts prefilled and written, steps, a call over several more tokens behind what is read back, steps again:
    each as the attention over the whole sequence, with the values that the cache holds."""
    N, H, KV, d, window, sinks = 3, 4, 2, 64, 24, 2
    lens, rows = [50, 7, 26], 26
    cache = torch.empty(2, 5, KV, rows, d, device="cuda").to(E4M3 if kind == "e4m3" else torch.bfloat16)
    scales = torch.empty(2, 5, KV, rows, device="cuda") if kind == "e4m3" else None
    slots = i32(4, 0, 2)
    total = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    q, k, v = (draw(i, 1, total, h, d) for i, h in enumerate((H, KV, KV)))
    gdn.swa_fwd(q, k, v, window, sinks, cu_tensor(cu))
    gdn.cache_write(cache, k, v, None, sinks, scales, slots, cu_tensor(cu))
    # every sequence's keys and values as the cache rounds them
    def rounded(x):
        if kind == "bf16":
            return host(x)
        flat = host(x).reshape(-1, d)
        return np.stack([np.multiply(*A.e4m3(r)) for r in flat]).reshape(x.shape)
    seen = [[rounded(x[0, a:b]) for x in (k, v)] for a, b in zip(cu, cu[1:])]
    lengths = i32(*lens)
    bound = 8 * HALF["bf16"]      # o: a mean of values of size 4, probabilities and o rounded once

    def step(seed):
        q, k, v = (draw(seed + i, N, h, d) for i, h in enumerate((H, KV, KV)))
        o = gdn.swa_step(cache, q, k, v, lengths, sinks, scales, slots)
        lengths.add_(1)
        for n in range(N):
            for s, x in zip((0, 1), (k, v)):
                seen[n][s] = np.concatenate([seen[n][s], rounded(x[n:n + 1])])
            want, _ = A.attention(host(q[n])[None, None], seen[n][0][None], seen[n][1][None], window, sinks)
            worst = np.abs(host(o[n]) - want[0, 0]).max()
            assert worst <= bound, (seed, n)

    for seed in range(100, 130, 10):
        step(seed)
    # several more tokens: keys are what is read back, then the new ones
    more = [5, 1, 30]
    cun = np.concatenate([[0], np.cumsum(more)]).tolist()
    have = [min(x, rows) for x in lengths.tolist()]
    cuk = np.concatenate([[0], np.cumsum(np.array(have) + more)]).tolist()
    kk, vv = (torch.empty(1, cuk[-1], KV, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gdn.cache_read(cache, lengths, sinks, scales, slots, cu_tensor(cuk), k=kk, v=vv)
    q, k, v = (draw(900 + i, 1, cun[-1], h, d) for i, h in enumerate((H, KV, KV)))
    for n in range(N):
        for to, x in ((kk, k), (vv, v)):
            to[0, cuk[n] + have[n]:cuk[n + 1]] = x[0, cun[n]:cun[n + 1]]
    o, _ = gdn.swa_fwd(q, kk, vv, window, sinks, cu_tensor(cun), cu_tensor(cuk))
    gdn.cache_write(cache, k, v, lengths, sinks, scales, slots, cu_tensor(cun))
    for n in range(N):
        part = slice(cun[n], cun[n + 1])
        full = [np.concatenate([s, host(x[0, part])]) for s, x in zip(seen[n], (k, v))]
        want, _ = A.attention(host(q[:, part]), full[0][None], full[1][None], window, sinks)
        worst = np.abs(host(o[:, part]) - want).max()
        assert worst <= bound, n
        seen[n] = [np.concatenate([s, rounded(x[0, part])]) for s, x in zip(seen[n], (k, v))]
    lengths += i32(*more)
    for seed in range(200, 220, 10):
        step(seed)


def test_fork_and_compaction():
    """A prompt's cache and scales forked and moved by state_move: every sequence gets the bits that it gets where
    nothing is moved."""
    KV, d, window, sinks, rows = 2, 32, 13, 1, 14
    cache = torch.empty(2, 6, KV, rows, d, device="cuda").to(E4M3)
    scales = torch.empty(2, 6, KV, rows, device="cuda")
    k, v = draw(1, 1, 20, KV, d), draw(2, 1, 20, KV, d)
    gdn.cache_write(cache, k, v, None, sinks, scales, i32(3))
    for x in (cache, scales):
        gdn.state_move(x, i32(3, 3), i32(0, 5), layers=True)

    def step(c, s, slots, t, who):
        q, k, v = (draw(50 + 3 * t + i, 3, h, d)[who].contiguous() for i, h in enumerate((4, KV, KV)))
        return gdn.swa_step(c, q, k, v, torch.full((len(who),), 20 + t, dtype=torch.int32, device="cuda"), sinks, s,
                            slots)

    still = cache.clone(), scales.clone()
    a = step(*still, i32(3, 0, 5), 0, [0, 1, 2])
    b = step(cache, scales, i32(3, 0, 5), 0, [0, 1, 2])
    assert torch.equal(a, b)
    for x in (cache, scales):               # the first sequence ends; the others move to slots 1 and 2
        gdn.state_move(x, i32(0, 5), i32(1, 2), layers=True)
    for t in range(1, 4):
        a = step(*still, i32(3, 0, 5), t, [0, 1, 2])
        b = step(cache, scales, i32(1, 2), t, [1, 2])
        assert torch.equal(a[1:], b)


def test_hybrid_steps_of_both_mixers():
    """One token through a gated delta layer and a windowed attention layer, as a stack alternates them."""
    N, H, d = 3, 2, 64
    state = torch.zeros(N, H, d, d, device="cuda")
    cache = torch.empty(2, N, H, 9, d, dtype=torch.bfloat16, device="cuda")
    lengths = i32(0, 0, 0)
    ks, vs = [], []
    for t in range(12):
        q, k, v = (draw(7 * t + i, N, H, d) for i in range(3))
        kn = torch.nn.functional.normalize(k.float(), dim=-1).bfloat16()
        mid = gdn.decode_step(state, q, kn, v, torch.full((N, H), -0.1, device="cuda"),
                              torch.full((N, H), 0.5, device="cuda"), out_dtype=torch.bfloat16)
        o = gdn.swa_step(cache, mid, k, mid, lengths, 1)
        lengths += 1
        ks.append(host(k)), vs.append(host(mid))
        kk, vv = np.stack(ks, 1), np.stack(vs, 1)
        want, _ = A.attention(host(mid)[:, None], kk, vv, 8, 1)
        worst = np.abs(host(o) - want[:, 0]).max()
        assert worst <= 4 * HALF["bf16"] * np.abs(vv).max()


def test_two_calls_at_once():
    """Two streams, each with its own tensors and workspaces."""
    sets = []
    for i in range(2):
        t = [draw(10 * i + j, 1, 700, h, 64) for j, h in enumerate((4, 2, 2, 4))]
        sets.append((t, cu_tensor([0, 100 + i, 700])))

    def run(t, c):
        o, lse = gdn.swa_fwd(*t[:3], 60, 3, c)
        return (o, lse, *gdn.swa_bwd(t[3], *t[:3], o, lse, 60, 3, c))

    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(run(*s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
