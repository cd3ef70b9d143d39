"""The operators around the attention kernels on the GPU, against their fp64 definitions.

Tolerances count roundings.  bf16 rounds by at most 2^-8 of the value, fp32 by 2^-24 (u below).
* Norm and rotation: y = r (z_a c - z_b s) in fp32.  The 128-term sum of squares has 12
  dependent steps (8 in a lane, 4 shuffles), rsqrt 2, the products and the rotation under 8:
  at most 32 u of |r z_a c| + |r z_b s|, then one rounding to bf16.
* Its backward: dx = r (t - x m), two such sums: 40 u of r (|t| + |x| M), M = r^2 mean|x t|;
  a gain's gradient adds its rows in a chain of fewer than 300 steps: 340 u of the sum of
  |dz x r|.
* Tree attention: the weights are rounded to bf16 before the product and O once after:
  2^-8 (|O| + A) with A = sum_j P_j |V_j|, and 2 % of that for the second order and the fp32
  steps.  LSE: a score is off by at most (d + 2) u of scale sum_c |q_c k_c|, and the sum of
  exponentials, its joins, the base-2 logarithm and the exponential by 600 u.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import workloads
from io_aware_softmax_b200 import (attn_bwd, attn_decode_paged, attn_decode_tree,
                                   attn_decode_tree_workspace_bytes, attn_fwd,
                                   attn_last_error_site, attn_page_tables,
                                   attn_qk_norm_rope, attn_qk_norm_rope_bwd,
                                   attn_qk_norm_rope_bwd_workspace_bytes, attn_qk_norm_rope_paged,
                                   attn_set_wait_limit_ns, device_status)
from tests.gpu_common import f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def randn(shape, seed, k=0, std=1.0):
    return workloads.randn_bf16(shape, seed, k, std).cuda()


def within(got, want, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4],
                           want[bad][:4])


# ------------------------------------------------------------------------- page tables

def check_tables(ctx, new, pool, table, page, T, used=None, parents=None, held=None):
    got = attn_page_tables(i32(ctx), i32(new), i32(pool), t := i32(table).reshape(len(ctx), -1),
                           page_size=page, num_tokens=T,
                           free_used=None if used is None else i32([used]),
                           parents=None if parents is None else i32(parents),
                           held_rows=None if held is None else i32(held))
    want = oracle.page_tables(ctx, new, pool, np.reshape(table, (len(ctx), -1)), page, T,
                              used or 0, parents, held)
    for g, w, name in zip((*got, t), want,
                          ("slots", "positions", "seq_lens", "offsets", "used", "table")):
        assert np.array_equal(g.cpu().numpy(), w), (name, g.cpu().numpy(), w)


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("B", [1, 2, 7, 255, 256, 257, 700])
def test_page_tables_random(page, B):
    rng = np.random.default_rng(B * 100 + page)
    P = 40
    ctx = rng.integers(-2, P * page + 3, B)
    new = rng.integers(-1, 3 * page + 2, B)
    table = rng.integers(0, 1000, (B, P))
    pool = rng.permutation(20 * B + 5)
    total = int(np.maximum(new, 0).sum())
    for T in (total, total + 13, max(total - 5, 0)):
        check_tables(ctx.tolist(), new.tolist(), pool.tolist(), table.tolist(), page, T)
    held = ctx + rng.integers(-3, 2 * page + 2, B)
    check_tables(ctx.tolist(), new.tolist(), pool.tolist(), table.tolist(), page, total,
                 held=held.tolist())


def test_page_tables_edges():
    check_tables([0], [0], [], [[]], 64, 0)                       # no room at all
    check_tables([0], [5], [], [[7, 7]], 4, 5)                    # an empty pool
    check_tables([5, 1], [9, 9], [1, 2, 3], [[0] * 4] * 2, 4, 18, used=2)
    check_tables([5, 1], [9, 9], [1, 2, 3], [[0] * 4] * 2, 4, 18, used=-4)
    check_tables([3, 2 ** 31 - 1], [2 ** 31 - 1, 2 ** 31 - 1], [1, 2, 3], [[0] * 4] * 2, 4, 40)
    check_tables([0] * 16384, [1] * 16384, list(range(16384)), [[-1]] * 16384, 64, 16384)
    # a page of the pool or of the table that is no page
    check_tables([4, 0], [4, 3], [-1, 6], [[-1, 0], [0, 0]], 4, 7)


@pytest.mark.parametrize("B", [2700, 2709, 2720, 2730, 2740, 4070, 4075, 4090, 4095, 4096])
def test_page_tables_sequences_that_fill_48_kb(B):
    # 12 bytes a sequence and the block's fixed part: below, at and above what a block has
    # without asking for more (in a process of its own: asking once is enough for all calls)
    code = f"""
import torch
from io_aware_softmax_b200 import attn_page_tables, device_status
e = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
for parents in (None, e([0] * {B})):
    slots, pos, lens, off, used = attn_page_tables(
        e([3] * {B}), e([1] * {B}), e([]), e([[7]] * {B}), page_size=64, num_tokens={B},
        parents=parents)
    assert (slots == 7 * 64 + 3).all() and (pos == 3).all() and (lens == 4).all()
    assert off.tolist() == list(range({B} + 1)) and used.item() == 0 and device_status() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr


def test_page_tables_no_sequences():
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    slots, pos, lens, off, used = attn_page_tables(
        e, e, e, e.reshape(0, 4), page_size=64, num_tokens=5, free_used=i32([3]))
    assert slots.tolist() == [-1] * 5 and pos.tolist() == [0] * 5
    assert off.tolist() == [0] and used.tolist() == [3] and lens.numel() == 0


@pytest.mark.parametrize("seed", range(3))
def test_page_tables_trees(seed):
    rng = np.random.default_rng(seed)
    new = rng.integers(0, 130, 9)
    parents = np.concatenate([rng.integers(-1, np.arange(n) + 2) for n in new] + [[0, 0]])
    ctx = rng.integers(0, 500, 9)
    check_tables(ctx.tolist(), new.tolist(), list(range(100)), [[0] * 20] * 9, 32,
                 len(parents), parents=parents.tolist())


def _parents(kind, n, rng):
    i = np.arange(n)
    if kind == "chain":
        return i - 1
    if kind == "near":
        return i - 1 - np.minimum(rng.integers(0, 3, n), i)
    if kind == "far":                       # anywhere before, across many chunks
        return rng.integers(-1, np.maximum(i, 1))
    if kind == "combs":                     # long lines that hang on early nodes, and bad entries
        p = i - 1
        at = rng.integers(0, n, n // 300 + 1)
        p[at] = rng.choice([-9, 0, 1, n, 2 ** 31 - 1], len(at))
        return p
    return np.full(n, -1)


@pytest.mark.parametrize("kind", ["chain", "near", "far", "combs", "none"])
@pytest.mark.parametrize("long", [255, 256, 257, 2048, 2049, 4096, 9001])
def test_page_tables_long_trees_beside_small_ones(kind, long):
    # sequences of one warp, of one chunk of a block, of several: small ones before and behind
    rng = np.random.default_rng(long)
    new = [3, 0, long, 60, 1, 300, long // 2 + 1, 17]
    parents = np.concatenate([_parents(kind if n > 20 else "near", n, rng) for n in new] + [[0]])
    ctx = rng.integers(0, 500, len(new))
    T = len(parents)
    for tokens in (T, T - 300):           # and cut within the last sequences
        check_tables(ctx.tolist(), new, list(range(T // 64 + 30)), [[0] * 160] * len(new), 64,
                     tokens, parents=parents[:tokens].tolist())


def test_page_tables_many_trees():
    # several sequences a warp, and long ones that share a block
    rng = np.random.default_rng(4)
    new = rng.integers(0, 12, 9000)
    new[rng.integers(0, 9000, 40)] = 400
    new[[5, 5 + 592, 5 + 1184]] = 3000
    parents = np.concatenate([_parents("near", int(n), rng) for n in new])
    check_tables([5] * 9000, new.tolist(), list(range(9999)), [[0] * 48] * 9000, 64, len(parents),
                 parents=parents.tolist())


def test_page_tables_time_goes_by_the_tokens_and_not_by_the_depth():
    # a chain of 8192 through parents beside small trees; a walk of every node to its root took
    # 270 times as long as the call without parents; 64 times leave room for noise
    new = [8192] + [40] * 16
    parents = np.concatenate([_parents("chain", n, None) for n in new])
    T = len(parents)
    args = (i32([100] * 17), i32(new), i32(list(range(400))), i32([[0] * 160] * 17))
    out = dict(slots=torch.empty(T, dtype=torch.int64, device="cuda"), positions=i32([0] * T),
               seq_lens=i32([0] * 17), token_offsets=i32([0] * 18), pages_used=i32([0]))

    def timed(p):
        attn_page_tables(*args, page_size=64, num_tokens=T, parents=p, **out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(10):
                attn_page_tables(*args, page_size=64, num_tokens=T, parents=p, **out)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        best = float("inf")
        for _ in range(5):
            a.record()
            graph.replay()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    assert timed(i32(parents)) <= 64 * timed(None)


@pytest.mark.parametrize("seed", range(4))
def test_page_tables_trees_after_rejected_drafts(seed):
    # the step after one whose drafts were taken back: held rows and parents together
    rng = np.random.default_rng(40 + seed)
    B = 11
    new = rng.integers(0, 70, B)
    parents = np.concatenate([rng.integers(-1, np.arange(n) + 1) for n in new] + [[-1] * 5])
    ctx = rng.integers(0, 400, B)
    held = ctx + rng.integers(-5, 80, B)
    table = rng.integers(100, 200, (B, 16))
    for T in (len(parents), len(parents) - 40):
        check_tables(ctx.tolist(), new.tolist(), list(range(60)), table.tolist(), 32, T, used=7,
                     parents=parents[:T].tolist(), held=held.tolist())


def test_page_tables_large_offsets():
    # slots past 2^31: a page number near 2^31 times its size
    slots, *_ = attn_page_tables(i32([0]), i32([65]), i32([2 ** 31 - 2, 2 ** 30]), i32([[0, 0]]),
                                 page_size=64, num_tokens=65)
    assert slots[0].item() == (2 ** 31 - 2) * 64 and slots[64].item() == 2 ** 30 * 64


# ----------------------------------------------------------------- norm and rotation

def rope(rows, rot, far=0):
    a = (np.arange(rows)[:, None] + far) * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


def prep_inputs(tokens, Hq, Hkv, d, rot, norm, seed, rows=600, std=1.0):
    x = randn((tokens, Hq + 2 * Hkv, d), seed, 0, std)
    w = (None, None)
    if norm:
        w = tuple((1 + 0.3 * randn((d,), seed, k).float()).bfloat16() for k in (1, 2))
    return x, w, rope(rows, rot) if rot else None


def prep_expected(x, w, table, pos, Hq, eps, inter):
    args = (f64(x), *(None if a is None else f64(a) for a in w),
            None if table is None else f64(table), pos)
    want = oracle.qk_norm_rope(*args, Hq, eps, inter)
    # what the roundings scale with: the same sums over absolute values
    mag = [np.abs(a) for a in oracle.qk_norm_rope(*args[:3], None, pos, Hq, eps, inter)]
    if table is not None and table.shape[1]:
        cs = np.abs(f64(table))
        for m in mag[:2]:
            rot = table.shape[1]
            lo, hi = oracle.serving._pairs(rot, inter)
            m[..., lo], m[..., hi] = m[..., lo] + m[..., hi], m[..., lo] + m[..., hi]
    return want, [BF * np.abs(o) + 32 * U * m + 2.0 ** -133 for o, m in zip(want, mag)]


def heads_first(t):      # [B, heads, N, d] -> [tokens, heads, d]
    return t.transpose(1, 2).reshape(-1, t.shape[1], t.shape[3])


PREP = [  # B, N, Hq, Hkv, d, rot, norm, interleaved
    (1, 1, 1, 1, 64, 64, True, False), (2, 37, 4, 2, 128, 128, True, False),
    (2, 37, 4, 2, 128, 128, True, True), (3, 65, 5, 1, 64, 32, True, False),
    (3, 65, 5, 1, 64, 32, True, True), (1, 130, 6, 3, 128, 16, False, True),
    (1, 130, 6, 3, 128, 48, False, False), (2, 9, 7, 7, 64, 0, True, False),
    (1, 300, 32, 8, 128, 64, True, False), (2, 5, 3, 2, 64, 64, False, False)]


@pytest.mark.parametrize("case", PREP)
@pytest.mark.parametrize("given", [False, True])
def test_qk_norm_rope(case, given):
    B, N, Hq, Hkv, d, rot, norm, inter = case
    x, w, table = prep_inputs(B * N, Hq, Hkv, d, rot, norm, N + d)
    rng = np.random.default_rng(N)
    pos = rng.integers(-3, 603, B * N) if given else np.tile(np.arange(N), B)
    q, k, v = attn_qk_norm_rope(x.view(B, N, -1, d), *w, table, num_q_heads=Hq, eps=1e-5,
                                positions=i32(pos).view(B, N) if given else None,
                                interleaved=inter)
    assert q.shape == (B, Hq, N, d) and k.shape == v.shape == (B, Hkv, N, d)
    want, bound = prep_expected(x, w, table, pos, Hq, 1e-5, inter)
    for got, o, e, name in zip((q, k, v), want, bound, "qkv"):
        within(heads_first(got), o, e, name)
    assert torch.equal(heads_first(v), x[:, Hq + Hkv:])
    assert device_status() == 0


def test_qk_norm_rope_values_of_every_size():
    # rows of zeros, tiny and large values; an infinity stays in its row
    x, w, table = prep_inputs(6, 2, 1, 128, 128, True, 5)
    x[0] = 0
    x[1] *= 2.0 ** -60
    x[2] *= 2.0 ** 40
    x[3, 0, 7] = float("inf")
    q, k, v = attn_qk_norm_rope(x.view(1, 6, 4, 128), *w, table, num_q_heads=2, eps=1e-6)
    ok = np.array([0, 1, 2, 4, 5])
    want, bound = prep_expected(x[ok], w, table, ok, 2, 1e-6, False)
    for got, o, e in zip((q, k, v), want, bound):
        within(heads_first(got)[ok], o, e, "sizes")
    assert not q[0, 0, 3].isfinite().all() and q[0, 1, 3].isfinite().all()


@pytest.mark.parametrize("case", PREP)
@pytest.mark.parametrize("given", [False, True])
def test_qk_norm_rope_bwd(case, given):
    B, N, Hq, Hkv, d, rot, norm, inter = case
    x, w, table = prep_inputs(B * N, Hq, Hkv, d, rot, norm, N + d + 1)
    rng = np.random.default_rng(N)
    pos = rng.integers(-3, 603, B * N) if given else np.tile(np.arange(N), B)
    g = [randn((B, h, N, d), 77, i) for i, h in enumerate((Hq, Hkv, Hkv))]
    dx, dwq, dwk = attn_qk_norm_rope_bwd(x.view(B, N, -1, d), *w, table, *g, eps=1e-5,
                                         positions=i32(pos).view(B, N) if given else None,
                                         interleaved=inter)
    gh = [f64(heads_first(t)) for t in g]
    wf = [None if a is None else f64(a) for a in w]
    tf = None if table is None else f64(table)
    want, wq, wk = oracle.qk_norm_rope_backward(f64(x), *wf, tf, pos, *gh, 1e-5, inter)
    mags, sums = [], []
    for lo, hi, wt, gg in ((0, Hq, wf[0], gh[0]), (Hq, Hq + Hkv, wf[1], gh[1])):
        m = np.abs(gg)
        if rot:
            a, b = oracle.serving._pairs(rot, inter)
            m[..., a], m[..., b] = m[..., a] + m[..., b], m[..., a] + m[..., b]
        if norm:
            xs = np.abs(f64(x)[:, lo:hi])
            r = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + 1e-5)
            t = m * np.abs(wt)
            sums.append((m * xs * r).sum((0, 1)))
            m = r * (t + xs * r * r * (xs * t).mean(-1, keepdims=True))
        mags.append(m)
    mag = np.concatenate([*mags, np.zeros_like(gh[2])], 1)
    within(dx.reshape(want.shape), want, BF * np.abs(want) + 40 * U * mag + 2.0 ** -133, "dqkv")
    if norm:
        within(dwq, wq, 340 * U * sums[0], "dq_weight")
        within(dwk, wk, 340 * U * sums[1], "dk_weight")
    else:
        assert dwq is None and dwk is None
    assert device_status() == 0


def test_qk_norm_rope_bwd_against_differences_and_the_same_twice():
    # the kernels' own forward, differenced in the direction of a large step in one value
    B, N, Hq, Hkv, d = 1, 40, 4, 2, 64
    x, w, table = prep_inputs(B * N, Hq, Hkv, d, 64, True, 9)
    x = x.view(B, N, -1, d)
    g = [randn((B, h, N, d), 78, i) for i, h in enumerate((Hq, Hkv, Hkv))]
    dx, dwq, dwk = attn_qk_norm_rope_bwd(x, *w, table, *g, eps=1e-5)
    again = attn_qk_norm_rope_bwd(x, *w, table, *g, eps=1e-5)
    assert torch.equal(dx, again[0]) and torch.equal(dwq, again[1]) and torch.equal(dwk, again[2])

    def loss(wq):
        out = attn_qk_norm_rope(x, wq, w[1], table, num_q_heads=Hq, eps=1e-5)
        return sum((f64(o) * f64(gg)).sum() for o, gg in zip(out, g))

    h = 2.0                       # the result is linear in a gain: only roundings remain
    for c in (0, 13, 63):
        up, down = w[0].clone(), w[0].clone()
        up[c], down[c] = w[0][c] + h, w[0][c] - h
        step = (up[c] - down[c]).item()
        diff = (loss(up) - loss(down)) / step
        # the outputs that move (this value and its partner): each rounded twice by 2^-8 of
        # about 4, times its gradient, independently over 2 N Hq values
        assert abs(diff - dwq[c].item()) <= 6 * BF * 4 * np.sqrt(2 * 2 * N * Hq) / step * 2
        assert abs(dwq[c].item()) > 0


def test_qk_norm_rope_bwd_many_blocks():
    # more rows than one wave of blocks takes: shares of many blocks and trips per warp
    B, N, Hq, Hkv, d = 2, 3000 + 5, 8, 2, 128
    x, w, table = prep_inputs(B * N, Hq, Hkv, d, 128, True, 21, rows=N)
    g = [randn((B, h, N, d), 79, i) for i, h in enumerate((Hq, Hkv, Hkv))]
    dx, dwq, dwk = attn_qk_norm_rope_bwd(x.view(B, N, -1, d), *w, table, *g)
    gh = [f64(heads_first(t)) for t in g]
    want, wq, wk = oracle.qk_norm_rope_backward(f64(x), f64(w[0]), f64(w[1]), f64(table),
                                                np.tile(np.arange(N), B), *gh, 1e-6)
    err = np.abs(f64(dx).reshape(want.shape) - want)
    assert np.linalg.norm(err) <= BF * np.linalg.norm(want)
    # chain of a thread's own rows, then at most 300 more steps; |dz x r| averages below 1.1
    for got, ref, h in ((dwq, wq, Hq), (dwk, wk, Hkv)):
        within(got, ref, 400 * U * 1.1 * B * N * h * np.ones(d), "gain")


def _bwd64(x, w, table, pos, g, eps):
    """dqkv, the gains' gradients, and what their roundings scale with, in 64 bits on the GPU (the
    halves' pairing, all of d rotated): x [T, H, d], g three of [T, heads, d]."""
    Hq, Hkv = g[0].shape[1], g[1].shape[1]
    c, s = table.double()[pos][:, None].chunk(2, -1)
    turn = lambda a, b, c, s: torch.cat([a * c + b * s, b * c - a * s], -1)  # noqa: E731
    dx, mag, gains, sums = [], [], [], []
    for lo, dy, gain in ((0, g[0], w[0]), (Hq, g[1], w[1])):
        xs, dy = x[:, lo:lo + dy.shape[1]].double(), dy.double()
        dz = turn(*dy.chunk(2, -1), c, s)
        a, b = dy.abs().chunk(2, -1)
        m = torch.cat([a + b, a + b], -1)
        r = (xs.square().mean(-1, keepdim=True) + eps).rsqrt()
        t = dz * gain.double()
        dx.append(r * (t - xs * r * r * (xs * t).mean(-1, keepdim=True)))
        gains.append((dz * xs * r).sum((0, 1)))
        sums.append((m * xs.abs() * r).sum((0, 1)))
        t = m * gain.double().abs()
        mag.append(r * (t + xs.abs() * r * r * (xs.abs() * t).mean(-1, keepdim=True)))
    dx.append(g[2].double())
    mag.append(torch.zeros_like(dx[-1]))
    return torch.cat(dx, 1), torch.cat(mag, 1), gains, sums


def _check_bwd(x, w, table, g, eps, tokens_at_once):
    """Every value of the backward for x [B, N, H, d] and the default positions."""
    B, N, H, d = x.shape
    dx, dwq, dwk = attn_qk_norm_rope_bwd(x, *w, table, *g, eps=eps)
    assert device_status() == 0
    gains, sums = [0, 0], [0, 0]
    for b in range(B):
        for n in range(0, N, tokens_at_once):
            at = slice(n, min(n + tokens_at_once, N))
            pos = torch.arange(at.start, at.stop, device="cuda")
            want, mag, gw, gs = _bwd64(x[b, at], w, table, pos,
                                       [t[b][:, at].transpose(0, 1) for t in g], eps)
            bad = ~((dx[b, at].double() - want).abs()
                    <= BF * want.abs() + 40 * U * mag + 2.0 ** -133)
            assert not bad.any(), (b, n, bad.nonzero()[:4].tolist())
            gains = [a + v for a, v in zip(gains, gw)]
            sums = [a + v for a, v in zip(sums, gs)]
    # a thread adds its share of the rows in one chain (8 warps a block, 256 / d rows a warp)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for got, want, s, t in ((dwq, gains[0], sums[0], g[0]), (dwk, gains[1], sums[1], g[1])):
        chain = 1.1 * B * N * t.shape[1] / (2 * sms * 8 * 256 / d)
        assert ((got.double() - want).abs() <= (chain + 340) * U * s).all()


@pytest.mark.parametrize("case", [
    # many trips of every warp through the ring of copies: 8 steps a chunk, a chunk of one head
    # behind a full one; the 8-step form with full chunks; 4 rows a warp; few heads
    (2, 4003, 17, 3, 128), (1, 6007, 32, 8, 128), (1, 9001, 40, 5, 64), (3, 5001, 3, 1, 64),
    (2, 4001, 13, 13, 128), (1, 7001, 6, 2, 128)])
def test_qk_norm_rope_bwd_every_value_over_many_trips(case):
    B, N, Hq, Hkv, d = case
    x, w, table = prep_inputs(B * N, Hq, Hkv, d, d, True, N, rows=N)
    g = [randn((B, h, N, d), 83, i) for i, h in enumerate((Hq, Hkv, Hkv))]
    _check_bwd(x.view(B, N, -1, d), w, table, g, 1e-6, 1024)


PAGED = [(1, 1, 1, 64, 64, 64, True, False), (16, 32, 8, 128, 64, 128, True, False),
         (77, 6, 2, 64, 128, 32, True, True), (40, 7, 1, 128, 192, 16, False, False),
         (33, 4, 4, 64, 1, 64, False, True), (129, 8, 2, 128, 5, 128, True, False)]


@pytest.mark.parametrize("case", PAGED)
def test_qk_norm_rope_paged(case):
    T, Hq, Hkv, d, page, rot, norm, inter = case
    x, w, table = prep_inputs(T, Hq, Hkv, d, rot, norm, T + d)
    pages = -(-T // page) + 2
    rng = np.random.default_rng(T)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[1], slots[3], slots[4] = -1, pages * page, 2 ** 40
    pos = rng.integers(0, 600, T)
    kp, vp = (randn((pages, Hkv, page, d), 31, i) for i in range(2))
    k0, v0 = kp.clone(), vp.clone()
    q = attn_qk_norm_rope_paged(x, *w, table, i32(pos), torch.from_numpy(slots).cuda(), kp, vp,
                                eps=1e-5, interleaved=inter)
    want, bound = prep_expected(x, w, table, pos, Hq, 1e-5, inter)
    within(q, want[0], bound[0], "q")
    here = (slots >= 0) & (slots < pages * page)
    at = slots[here]
    touched = torch.zeros((pages, page), dtype=torch.bool)
    touched[at // page, at % page] = True
    for got, before, i in ((kp, k0, 1), (vp, v0, 2)):
        rows = got.cpu()[at // page, :, at % page]
        within(rows, want[i][here], bound[i][here], "kv"[i - 1])
        keep = ~touched[:, None, :, None].expand(got.shape)
        assert torch.equal(got.cpu()[keep], before.cpu()[keep])
    assert device_status() == 0


def test_prepared_inputs_train_through_attention():
    # projection output -> norm and rotation -> attention -> back to the projection's gradient:
    # the gradient is the directional derivative of the same chain in fp64
    B, N, Hq, Hkv, d = 1, 96, 4, 2, 64
    x, w, table = prep_inputs(B * N, Hq, Hkv, d, 64, True, 50, rows=N)
    x = x.view(B, N, -1, d)
    q, k, v = attn_qk_norm_rope(x, *w, table, num_q_heads=Hq)
    o, lse = attn_fwd(q, k, v, mask="causal")
    do = randn((B, Hq, N, d), 51)
    dq, dk, dv = attn_bwd(q, k, v, o, lse, do, mask="causal")
    dx, dwq, dwk = attn_qk_norm_rope_bwd(x, *w, table, dq, dk, dv)
    assert device_status() == 0
    pos = np.arange(N)
    xs = f64(x).reshape(N, -1, d)
    qq, kk, vv = oracle.qk_norm_rope(xs, f64(w[0]), f64(w[1]), f64(table), pos, Hq, 1e-6)
    swap = lambda a: a.transpose(1, 0, 2)[None]  # noqa: E731
    g = oracle.attention_backward(swap(qq), swap(kk), swap(vv), f64(do), mask_kind=1)
    back = [a[0].transpose(1, 0, 2) for a in g]
    want, wq, wk = oracle.qk_norm_rope_backward(xs, f64(w[0]), f64(w[1]), f64(table), pos, *back,
                                                1e-6)
    # attn_bwd's own bounds (1.5e-2 of the largest, 4e-3 of the mean) and the roundings here
    err = np.abs(f64(dx).reshape(want.shape) - want)
    assert err.max() <= 1.5e-2 * np.abs(want).max() + BF * np.abs(want).max()
    assert err.mean() <= (4e-3 + BF) * np.abs(want).mean()
    for got, ref in ((dwq, wq), (dwk, wk)):
        assert np.abs(f64(got) - ref).max() <= 1.5e-2 * np.abs(ref).max()


# --------------------------------------------------------------------- tree attention

def tree_inputs(lens, n, Hq, Hkv, d, page, seed, std=1.0, spare_rows=0, branch=4):
    rng = np.random.default_rng(seed)
    T = sum(n) + spare_rows
    held = [-(-max(L, 0) // page) for L in lens]
    P = max(max(held), 1)
    pages = sum(held) + 2
    q = randn((T, Hq, d), seed, 0, std)
    kp = randn((pages, Hkv, page, d), seed, 1, std)
    vp = randn((pages, Hkv, page, d), seed, 2)
    order = rng.permutation(pages)
    table = np.full((len(lens), P), 2 ** 30, np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    parents = [max(-1, i - 1 - int(rng.integers(branch))) for m in n for i in range(m)]
    offsets = np.concatenate([[0], np.cumsum(n)])
    return q, kp, vp, table, offsets, np.array(parents + [0] * spare_rows)


def check_tree(lens, n, Hq, Hkv, d, page, seed, chain=False, std=1.0, max_nodes=None, scale=None,
               parents=None, **kw):
    q, kp, vp, table, offsets, par = tree_inputs(lens, n, Hq, Hkv, d, page, seed, std)
    par = None if chain else par if parents is None else np.array(parents)
    nodes = max(n) if max_nodes is None else max_nodes
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    attn_decode_tree(q, kp, vp, i32(table), i32(lens), i32(offsets), max_nodes=nodes, scale=scale,
                     parents=None if chain else i32(par), out=out, lse=lse, **kw)
    assert device_status() == 0
    O, L, A = oracle.decode_tree(f64(q), f64(kp), f64(vp), table, lens, offsets, par, scale, nodes)
    mine = ~np.isnan(L)
    within(f64(out)[mine], O[mine], 1.02 * BF * (np.abs(O) + A)[mine] + 2.0 ** -133, "O")
    got = f64(lse)
    none = np.isneginf(L)
    assert np.array_equal(np.isneginf(got), none)
    length = lambda x: np.linalg.norm(f64(x), axis=-1).max(initial=0)  # noqa: E731
    s = (scale or d ** -0.5) * length(q) * length(kp)
    some = mine & ~none
    within(got[some], L[some], U * ((d + 2) * s + 600 + np.abs(L[some])), "LSE")
    assert (f64(out)[~mine] == 7).all() and (got[~mine] == 7).all()
    return out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [64, 128, 192])
def test_tree_lengths(d, page):
    n = [1, 2, 5, 8, 3, 7, 1, 8, 4]
    lens = [1, 2, 63, 64, 65, 128, 129, 700, 1025]
    check_tree(lens, n, 8, 2, d, page, seed=d + page)
    check_tree(lens, n, 8, 2, d, page, seed=d + page + 1, chain=True)


@pytest.mark.parametrize("G,nodes", [(1, 1), (1, 128), (2, 65), (3, 43), (3, 40), (4, 32), (4, 33),
                                     (4, 64), (5, 26), (7, 19), (8, 16), (8, 17), (16, 8), (16, 9),
                                     (16, 40), (12, 128)])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_group_sizes_and_widths(G, nodes, d):
    n = [nodes, max(1, nodes // 3), nodes - 1, 1]
    check_tree([m + c for m, c in zip(n, (300, 0, 517, 40))], n, 2 * G, 2, d, 64, seed=G * nodes)


def test_tree_nodes_across_a_tile_and_a_page():
    # drafted rows that begin in one 128-key tile and end in the next, at every offset near it
    for ctx in (60, 100, 120, 126, 127, 128, 129, 250):
        check_tree([ctx + 90, ctx + 128], [90, 128], 2, 1, 64, 64, seed=ctx)


def test_tree_empty_sequences_short_lengths_and_rows_left_alone():
    check_tree([100, 0, 300, 50, 0], [4, 0, 0, 3, 0], 4, 2, 128, 64, seed=1)
    # lengths below the number of drafted tokens, zero and negative
    check_tree([3, 0, -7, 200], [5, 4, 2, 6], 4, 2, 128, 64, seed=2)
    # only the first max_nodes of a longer sequence
    check_tree([90, 200], [30, 9], 4, 2, 64, 64, seed=3, max_nodes=7)
    check_tree([190, 200], [100, 9], 4, 2, 64, 64, seed=4, max_nodes=70)
    check_tree([1000], [200], 2, 2, 64, 64, seed=5, max_nodes=128)
    # nothing drafted at all
    check_tree([100, 30], [0, 0], 4, 2, 64, 64, seed=6, max_nodes=4)


def test_tree_bad_parents_count_as_none():
    check_tree([80], [8], 4, 2, 64, 64, seed=7, parents=[5, 1, 0, -9, 2, 900, 4, 7])
    deep = list(range(-1, 127))
    check_tree([700], [128], 1, 1, 128, 64, seed=8, parents=deep)


def test_tree_large_scores_and_scale():
    check_tree([900, 333], [9, 12], 8, 2, 128, 64, seed=9, std=3.0)
    check_tree([900, 333], [9, 12], 8, 2, 64, 64, seed=10, scale=0.5)


def test_tree_many_short_sequences():
    rng = np.random.default_rng(11)
    n = rng.integers(0, 6, 500).tolist()
    lens = [m + int(c) for m, c in zip(n, rng.integers(0, 300, 500))]
    check_tree(lens, n, 4, 2, 64, 64, seed=11)


def test_tree_one_long_sequence_over_many_ctas():
    check_tree([20011], [11], 4, 1, 128, 64, seed=12)
    check_tree([20011, 5], [70, 5], 4, 1, 128, 128, seed=13)


def test_tree_rows_behind_the_last_sequence_and_garbage_past_the_end():
    # rows of q past the last offset stay; what pages hold past a sequence's end may be anything
    q, kp, vp, table, offsets, par = tree_inputs([70, 150], [5, 9], 8, 2, 128, 64, 14, spare_rows=6)
    O, L, A = oracle.decode_tree(f64(q), f64(kp), f64(vp), table, [70, 150], offsets, par)
    for p in (kp, vp):
        p[int(table[0, 1]), :, 6:] = float("nan")
        p[int(table[1, 2]), :, 22:] = float("inf")
    out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 3.0, device="cuda")
    attn_decode_tree(q, kp, vp, i32(table), i32([70, 150]), i32(offsets), max_nodes=9,
                     parents=i32(par), out=out, lse=lse)
    assert device_status() == 0
    within(f64(out)[:14], O[:14], 1.02 * BF * (np.abs(O) + A)[:14], "O")
    assert (out[14:] == 3).all() and (lse[14:] == 3).all() and lse[:14].isfinite().all()


def test_tree_garbage_past_the_end_of_long_sequences():
    # the last tile comes many rounds of the tile ring after the first
    lens, n = [3000, 1777, 2600], [6, 3, 1]
    q, kp, vp, table, offsets, par = tree_inputs(lens, n, 4, 1, 128, 64, 17)
    O, L, A = oracle.decode_tree(f64(q), f64(kp), f64(vp), table, lens, offsets, par)
    for b, length in enumerate(lens):
        for p in (kp, vp):
            p[int(table[b, length // 64]), :, length % 64:] = float("nan")
    out, lse = attn_decode_tree(q, kp, vp, i32(table), i32(lens), i32(offsets), max_nodes=6,
                                parents=i32(par))
    assert device_status() == 0
    within(out, O, 1.02 * BF * (np.abs(O) + A), "O")
    assert np.abs(f64(lse) - L).max() <= 1e-4


def test_tree_values_that_are_no_numbers_stay_with_the_rows_that_see_them():
    lens, n = [700, 2000], [6, 5]
    q, kp, vp, table, offsets, _ = tree_inputs(lens, n, 4, 2, 64, 64, 18)
    par = np.array([-1, 0, 0, 1, 2, -1, -1, 0, 0, 1, 2])
    q[7, 1] = float("nan")                      # a query row: sequence 1, node 1, head 1
    q[9, 2, 5] = float("inf")
    k_row = 700 - 6 + 2                         # the key of sequence 0's node 2, KV head 0
    kp[int(table[0, k_row // 64]), 0, k_row % 64, 3] = float("nan")
    bad = np.zeros((11, 4), bool)
    bad[7, 1] = bad[9, 2] = True
    bad[[2, 4], :2] = True                      # node 2 and its descendant see that key
    out, lse = attn_decode_tree(q, kp, vp, i32(table), i32(lens), i32(offsets), max_nodes=6,
                                parents=i32(par))
    assert device_status() == 0
    assert np.array_equal(np.isnan(f64(lse)), bad)
    assert np.isnan(f64(out)[bad]).all()
    q, kp = torch.nan_to_num(q, posinf=1.0), torch.nan_to_num(kp)
    O, L, A = oracle.decode_tree(f64(q), f64(kp), f64(vp), table, lens, offsets, par)
    within(f64(out)[~bad], O[~bad], 1.02 * BF * (np.abs(O) + A)[~bad], "O")
    assert np.abs(f64(lse) - L)[~bad].max() <= 1e-4


@pytest.mark.parametrize("d,Hq,nodes", [(64, 4, 7), (128, 4, 7), (64, 16, 40), (128, 16, 40),
                                        (128, 2, 120)])
def test_tree_values_that_are_no_numbers_in_hidden_rows(d, Hq, nodes):
    # infinities and NaN in K and V of drafted rows reach the nodes that see them and no other:
    # whole and cut sequences, rows of one tile and of two, few query rows and many
    lens = [nodes, 100 + nodes, 128 + nodes // 2, 3000 + nodes, 77]
    n = [nodes, nodes, nodes // 2, nodes, 3]
    q, kp, vp, table, offsets, par = tree_inputs(lens, n, Hq, 2, d, 64, d + nodes, branch=3)
    rng = np.random.default_rng(nodes)
    for b, (length, m) in enumerate(zip(lens[:4], n)):
        for cache, value in ((vp, "nan"), (vp, "inf"), (vp, "-inf"), (kp, "nan")):
            for _ in range(2):
                row = length - m + int(rng.integers(m // 2, m))
                cache[int(table[b, row // 64]), int(rng.integers(2)), row % 64,
                      int(rng.integers(d))] = float(value)
    with np.errstate(invalid="ignore"):
        O, L, A = oracle.decode_tree(f64(q), f64(kp), f64(vp), table, lens, offsets, par)
    assert np.isnan(O).any() and np.isinf(O).any() and np.isfinite(O).mean() > 0.3
    out, lse = attn_decode_tree(q, kp, vp, i32(table), i32(lens), i32(offsets), max_nodes=nodes,
                                parents=i32(par))
    assert device_status() == 0
    got, fin = f64(out), np.isfinite(O)
    assert np.array_equal(np.isnan(got), np.isnan(O)) and np.array_equal(got[np.isinf(O)],
                                                                         O[np.isinf(O)])
    # A is not finite beside an infinity of the same row's sum: |V| up to 6 bounds it there
    bound = 1.02 * BF * (np.abs(O) + np.where(np.isfinite(A), A, 6.0))
    within(got[fin], O[fin], bound[fin], "O")
    ok = np.isfinite(L)
    assert np.array_equal(np.isfinite(f64(lse)), ok) and np.abs(f64(lse) - L)[ok].max() <= 1e-4


def test_tree_cache_past_32_bit_offsets():
    # 2.6 G values a cache: the sequences' pages lie at its end and its beginning
    pages, Hkv, page, d = 40000, 8, 64, 128
    kp, vp = (torch.empty((pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    table = np.array([[pages - 1, 0, pages - 3], [1, pages - 2, 20000]])
    small = [randn((6, Hkv, page, d), 91, i) for i in range(2)]
    for big, few in zip((kp, vp), small):
        big[torch.from_numpy(table.reshape(-1)).cuda()] = few
    q = randn((9, 16, d), 92)
    lens, offsets = [170, 130], [0, 5, 9]
    out, lse = attn_decode_tree(q, kp, vp, i32(table), i32(lens), i32(offsets), max_nodes=5)
    assert device_status() == 0
    O, L, A = oracle.decode_tree(f64(q), f64(small[0]), f64(small[1]), np.arange(6).reshape(2, 3),
                                 lens, offsets)
    within(out, O, 1.02 * BF * (np.abs(O) + A), "O")
    assert np.abs(f64(lse) - L).max() <= 1e-4
    # and written there: slots of the last page and of the first
    x, w, rp = prep_inputs(4, 16, Hkv, d, 128, True, 93)
    slots = np.array([(pages - 1) * page + 63, 0, pages * page - 64, 5])
    q = attn_qk_norm_rope_paged(x, *w, rp, i32([7, 8, 9, 10]), torch.from_numpy(slots).cuda(), kp,
                                vp, eps=1e-5)
    want, bound = prep_expected(x, w, rp, [7, 8, 9, 10], 16, 1e-5, False)
    within(q, want[0], bound[0], "q")
    for cache, o, e in ((kp, want[1], bound[1]), (vp, want[2], bound[2])):
        sl = torch.from_numpy(slots).cuda()
        within(cache[sl // page, :, sl % page], o, e, "cache")


def test_qk_norm_rope_past_32_bit_offsets():
    # 2.3 G values in and out; tokens of both ends are checked, forward and backward
    B, N, Hq, Hkv, d = 3, 61440 + 3, 64, 16, 128
    x = torch.randn((B, N, Hq + 2 * Hkv, d), device="cuda", dtype=torch.bfloat16)
    assert x.numel() > 2 ** 31
    w = tuple((1 + 0.3 * randn((d,), 95, k).float()).bfloat16() for k in (1, 2))
    table = rope(N, 64)
    q, k, v = attn_qk_norm_rope(x, *w, table, num_q_heads=Hq, eps=1e-5)
    at = np.array([0, 1, N - 2, N - 1])
    for b in (0, B - 1):
        few = x[b, at].contiguous()
        want, bound = prep_expected(few, w, table, at, Hq, 1e-5, False)
        for got, o, e, name in zip((q, k, v), want, bound, "qkv"):
            within(got[b][:, at].transpose(0, 1), o, e, name)
    dx, _, _ = attn_qk_norm_rope_bwd(x, *w, table, q, k, v, eps=1e-5)
    for b in (0, B - 1):
        few = f64(x[b, at])
        g = [f64(t[b][:, at].transpose(0, 1)) for t in (q, k, v)]
        want, _, _ = oracle.qk_norm_rope_backward(few, f64(w[0]), f64(w[1]), f64(table), at, *g,
                                                  1e-5)
        # dy = y here, so t and x M nearly cancel: fp32 leaves 40 u of the terms, which are
        # below 16 (gains below 2, |y| below 8)
        within(dx[b, at], want, BF * np.abs(want) + 40 * U * 32, "dqkv")


def test_qk_norm_rope_bwd_every_value_past_32_bit_offsets():
    B, N, Hq, Hkv, d = 3, 61440 + 3, 64, 16, 128
    gen = torch.Generator(device="cuda").manual_seed(96)
    rand = lambda *s: torch.randn(s, device="cuda", dtype=torch.bfloat16,  # noqa: E731
                                  generator=gen)
    x = rand(B, N, Hq + 2 * Hkv, d)
    assert x.numel() > 2 ** 31
    w = tuple((1 + 0.3 * randn((d,), 97, k).float()).bfloat16() for k in (1, 2))
    g = [rand(B, h, N, d) for h in (Hq, Hkv, Hkv)]
    _check_bwd(x, w, rope(N, d), g, 1e-6, 4096)


def test_tree_pages_outside_the_cache_read_zeros():
    q, kp, vp, table, offsets, par = tree_inputs([200, 100], [3, 4], 4, 2, 64, 64, 15)
    table[0, 1], table[1, 0] = -1, kp.shape[0]
    out, lse = attn_decode_tree(q, kp, vp, i32(table), i32([200, 100]), i32(offsets), max_nodes=4,
                                parents=i32(par))
    assert device_status() == 0
    O, L, A = oracle.decode_tree(f64(q), f64(kp), f64(vp), table, [200, 100], offsets, par)
    within(out, O, 1.02 * BF * (np.abs(O) + A), "O")
    assert np.abs(f64(lse) - L).max() <= 1e-4
    # a cache without a page
    out, lse = attn_decode_tree(q, kp[:0], vp[:0], i32(table), i32([200, 100]), i32(offsets),
                                max_nodes=4)
    assert device_status() == 0 and not out.any() and lse.isneginf().all()


def test_tree_of_one_node_is_the_paged_decode():
    q, kp, vp, table, offsets, _ = tree_inputs([900, 64, 1], [1, 1, 1], 8, 2, 128, 64, 16)
    o1, l1 = attn_decode_tree(q, kp, vp, i32(table), i32([900, 64, 1]), i32(offsets), max_nodes=1)
    o2, l2 = attn_decode_paged(q.unsqueeze(2), kp, vp, i32(table), i32([900, 64, 1]))
    assert device_status() == 0
    # the two kernels round the weights alike but at other maxima
    assert (o1 - o2.squeeze(2)).abs().max().item() <= 2e-2
    assert (l1 - l2.squeeze(2)).abs().max().item() <= 1e-4


def test_tree_calls_back_to_back_on_one_workspace():
    # each call's kernels are launched while those of the call before still read the workspace:
    # cut segments, other lengths, offsets, batch sizes and widths, nothing else between
    shapes = [([3000, 1777, 20, 2600], [6, 9, 3, 1], 9), ([9000], [7], 9),
              ([40, 5000, 700], [40, 31, 40], 40), ([130] * 30, [2] * 30, 9),
              ([4000, 0, 4100, 60], [33, 0, 40, 12], 64), ([12000, 11], [1, 4], 4)]
    calls, bytes_ = [], 0
    for i, (lens, n, nodes) in enumerate(shapes):
        q, kp, vp, table, offsets, par = tree_inputs(lens, n, 16, 4, 128, 64, 200 + i)
        calls.append(((q, kp, vp, i32(table), i32(lens), i32(offsets)),
                      dict(max_nodes=nodes, parents=i32(par))))
        bytes_ = max(bytes_, attn_decode_tree_workspace_bytes(len(lens), 16, 4, nodes, 128))
    ws = torch.empty(bytes_, dtype=torch.uint8, device="cuda")
    alone = []
    for (args, kw), (lens, n, nodes) in zip(calls, shapes):
        o, lse = attn_decode_tree(*args, **kw)
        torch.cuda.synchronize()
        O, L, A = oracle.decode_tree(*(f64(t) for t in args[:3]), args[3].cpu().numpy(), lens,
                                     args[5].tolist(), kw["parents"].tolist())
        within(o, O, 1.02 * BF * (np.abs(O) + A), "O")
        assert np.abs(f64(lse) - L).max(initial=0) <= 1e-4
        alone.append((o, lse))
    order = np.random.default_rng(0).integers(0, len(calls), 60).tolist()
    outs = [tuple(torch.full_like(t, 7) for t in alone[i]) for i in order]

    def run():
        for i, (o, lse) in zip(order, outs):
            args, kw = calls[i]
            attn_decode_tree(*args, **kw, out=o, lse=lse, workspace=ws)

    def check():
        torch.cuda.synchronize()
        assert device_status() == 0
        for k, (i, got) in enumerate(zip(order, outs)):
            for a, b in zip(got, alone[i]):
                assert torch.equal(a, b), (k, i)
                a.fill_(7)

    run()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        graph.replay()
        check()


def test_tree_replayed_with_far_fewer_nodes_than_the_graph_was_captured_for():
    B, most, T = 5, 100, 320
    q, kp, vp, table, _, _ = tree_inputs([700] * B, [1] * B, 8, 2, 128, 64, 19,
                                         spare_rows=T - B)
    lens, offsets, parents = i32([0] * B), i32([0] * (B + 1)), i32([-1] * T)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    ws = torch.empty(attn_decode_tree_workspace_bytes(B, 8, 2, most, 128), dtype=torch.uint8,
                     device="cuda")
    args = (q, kp, vp, i32(table), lens, offsets)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn_decode_tree(*args, max_nodes=most, parents=parents, out=out, lse=lse, workspace=ws)
    rng = np.random.default_rng(19)
    for n in ([1, 1, 1, 1, 1], [4, 0, 7, 2, 5], [100, 3, 0, 33, 100], [0] * 5, [32, 33, 31, 64, 1]):
        L = [int(v) for v in rng.integers(100, 700, B)]
        off = np.concatenate([[0], np.cumsum(n)])
        par = [max(-1, i - 1 - int(rng.integers(3))) for m in n for i in range(m)]
        for t, v in ((lens, L), (offsets, off), (parents, par + [0] * (T - len(par)))):
            t.copy_(i32(v))
        out.fill_(7), lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert device_status() == 0
        m = int(off[-1])
        O, W, A = oracle.decode_tree(f64(q), f64(kp), f64(vp), table, L, off,
                                     par + [0] * (T - len(par)))
        within(f64(out)[:m], O[:m], 1.02 * BF * (np.abs(O) + A)[:m], "O")
        assert np.abs(f64(lse)[:m] - W[:m]).max(initial=0) <= 1e-4
        assert (out[m:] == 7).all() and (lse[m:] == 7).all()


# ------------------------------------------------------------------- a step of serving

def _step(s, o):
    """One verification step on preallocated buffers: tables, cache write, attention."""
    attn_page_tables(s["ctx"], s["new"], s["free"], s["table"], page_size=64,
                     num_tokens=s["qkv"].shape[0], parents=s["parents"], free_used=s["used"],
                     slots=o["slots"], positions=o["pos"], seq_lens=o["lens"],
                     token_offsets=o["off"], pages_used=o["used"])
    attn_qk_norm_rope_paged(s["qkv"], s["wq"], s["wk"], s["rope"], o["pos"], o["slots"], s["k"],
                            s["v"], q=o["q"])
    attn_decode_tree(o["q"], s["k"], s["v"], s["table"], o["lens"], o["off"], max_nodes=9,
                     parents=s["parents"], out=o["out"], lse=o["lse"], workspace=o["ws"])


def _step_state(seed):
    rng = np.random.default_rng(seed)
    ctx, new = rng.integers(0, 400, 5), rng.integers(1, 10, 5)
    ctx[2] = 0
    T, Hq, Hkv, d = 48, 4, 2, 64
    pool = rng.permutation(60)
    table = np.full((5, 8), -1)
    used = 3
    for b in range(5):
        for p in range(-(-int(ctx[b]) // 64)):
            table[b, p] = pool[used]
            used += 1
    parents = [max(-1, i - 1 - int(rng.integers(3))) for m in new for i in range(m)]
    parents += [-1] * (T - len(parents))
    x, w, rp = prep_inputs(T, Hq, Hkv, d, 64, True, seed)
    return dict(ctx=i32(ctx), new=i32(new), free=i32(pool), table=i32(table), used=i32([used]),
                parents=i32(parents), qkv=x, wq=w[0], wk=w[1], rope=rp,
                k=randn((60, Hkv, 64, d), seed, 5), v=randn((60, Hkv, 64, d), seed, 6))


def _step_outputs():
    e = lambda shape, t: torch.zeros(shape, dtype=t, device="cuda")  # noqa: E731
    return dict(slots=e(48, torch.int64), pos=e(48, torch.int32), lens=e(5, torch.int32),
                off=e(6, torch.int32), used=e(1, torch.int32), q=e((48, 4, 64), torch.bfloat16),
                out=e((48, 4, 64), torch.bfloat16), lse=e((48, 4), torch.float32),
                ws=e(attn_decode_tree_workspace_bytes(5, 4, 2, 9, 64), torch.uint8))


def test_a_verification_step_against_the_definitions():
    s, o = _step_state(60), _step_outputs()
    k0, v0 = f64(s["k"]), f64(s["v"])
    ctx, new, par = (s[n].tolist() for n in ("ctx", "new", "parents"))
    want = oracle.page_tables(ctx, new, s["free"].tolist(), s["table"].cpu().numpy(), 64, 48,
                              s["used"].item(), par)
    _step(s, o)
    assert device_status() == 0
    for n, w in zip(("slots", "pos", "lens", "off", "used"), want):
        assert np.array_equal(o[n].cpu().numpy(), w), n
    assert np.array_equal(s["table"].cpu().numpy(), want[5])
    slots, pos = want[0], want[1]
    heads, bound = prep_expected(s["qkv"], (s["wq"], s["wk"]), s["rope"], pos, 4, 1e-6, False)
    within(o["q"], heads[0], bound[0], "q")
    for page, before, x, e in ((s["k"], k0, heads[1], bound[1]), (s["v"], v0, heads[2], bound[2])):
        t = np.nonzero(slots >= 0)[0]
        within(f64(page)[slots[t] // 64, :, slots[t] % 64], x[t], e[t], "cache")
    # the attention of what was written
    O, L, A = oracle.decode_tree(f64(o["q"]), f64(s["k"]), f64(s["v"]), want[5], want[2], want[3],
                                 par)
    T = want[3][-1]
    within(f64(o["out"])[:T], O[:T], 1.02 * BF * (np.abs(O) + A)[:T] + 2.0 ** -133, "O")
    assert np.abs(f64(o["lse"])[:T] - L[:T]).max() <= 1e-4
    assert not o["out"][T:].any()


def test_the_step_captured_and_replayed():
    s, eager, cap = _step_state(61), _step_outputs(), _step_outputs()
    _step(s, eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(s, cap)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(s, cap)
    for seed in (61, 62, 63):          # lengths, tables and trees of other steps, in place
        new = _step_state(seed)
        for n in s:
            s[n].copy_(new[n])
        fresh = _step_outputs()
        _step(new, fresh)
        for n in ("out", "lse", "q"):
            cap[n].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert device_status() == 0
        for n in fresh:
            if n != "ws":
                assert torch.equal(cap[n], fresh[n]), n
        assert torch.equal(s["k"], new["k"]) and torch.equal(s["table"], new["table"])


def test_backward_captured_and_replayed():
    B, N, Hq, Hkv, d = 2, 70, 4, 2, 128
    x, w, table = prep_inputs(B * N, Hq, Hkv, d, 128, True, 70, rows=N)
    x = x.view(B, N, -1, d)
    g = [randn((B, h, N, d), 71, i) for i, h in enumerate((Hq, Hkv, Hkv))]
    out = dict(dqkv=torch.empty_like(x), dq_weight=torch.empty(d, device="cuda"),
               dk_weight=torch.empty(d, device="cuda"),
               workspace=torch.empty(attn_qk_norm_rope_bwd_workspace_bytes(d), dtype=torch.uint8,
                                     device="cuda"))
    want = attn_qk_norm_rope_bwd(x, *w, table, *g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn_qk_norm_rope_bwd(x, *w, table, *g, **out)
    graph.replay()
    for a, b in zip(want, (out["dqkv"], out["dq_weight"], out["dk_weight"])):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    states = [_step_state(80 + i) for i in range(2)]
    want = []
    for s in states:
        fresh = {n: t.clone() for n, t in s.items()}
        o = _step_outputs()
        _step(fresh, o)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [_step_outputs() for _ in states]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, st in zip(states, got, streams):
            with torch.cuda.stream(st):
                _step(s, o)
    torch.cuda.synchronize()
    assert device_status() == 0
    for a, b in zip(got, want):
        for n in a:
            if n != "ws":
                assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("nodes", [9, 40])
def test_a_wait_that_runs_out_is_reported_and_later_calls_run(nodes):
    # caches long enough that every CTA waits for many copies from memory: the device timer
    # advances in steps of up to a microsecond, and only a wait that sees it move runs out
    lens, n = [60000, 45000, 20], [nodes, 7, 3]
    q, kp, vp, table, offsets, par = tree_inputs(lens, n, 16, 4, 128, 64, 90)
    args = (q, kp, vp, i32(table), i32(lens), i32(offsets))
    want = attn_decode_tree(*args, max_nodes=nodes, parents=i32(par))
    assert device_status() == 0
    attn_set_wait_limit_ns(1)
    try:
        attn_decode_tree(*args, max_nodes=nodes, parents=i32(par))
        assert device_status() == -5
        assert attn_last_error_site() > 200
    finally:
        attn_set_wait_limit_ns(0)
    again = attn_decode_tree(*args, max_nodes=nodes, parents=i32(par))
    assert device_status() == 0
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_calls_on_a_given_stream():
    # the whole call, its allocations too, belongs to the stream that is given
    s = _step_state(85)
    fresh = {n: t.clone() for n, t in s.items()}
    want = _step_outputs()
    _step(fresh, want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    slots, pos, lens, off, used = attn_page_tables(
        s["ctx"], s["new"], s["free"], s["table"], page_size=64, num_tokens=48,
        free_used=s["used"], parents=s["parents"], stream=st)
    q = attn_qk_norm_rope_paged(s["qkv"], s["wq"], s["wk"], s["rope"], pos, slots, s["k"], s["v"],
                                stream=st)
    o, lse = attn_decode_tree(q, s["k"], s["v"], s["table"], lens, off, max_nodes=9,
                              parents=s["parents"], stream=st)
    x = s["qkv"].view(1, 48, 8, 64)
    qq, kk, vv = attn_qk_norm_rope(x, s["wq"], s["wk"], s["rope"], num_q_heads=4, stream=st)
    dx, dwq, dwk = attn_qk_norm_rope_bwd(x, s["wq"], s["wk"], s["rope"], qq, kk, vv, stream=st)
    st.synchronize()
    assert device_status() == 0
    n = int(off[-1])
    assert torch.equal(q, want["q"]) and torch.equal(o[:n], want["out"][:n])
    assert torch.equal(slots, want["slots"]) and torch.equal(s["k"], fresh["k"])
    again = attn_qk_norm_rope_bwd(x, s["wq"], s["wk"], s["rope"], qq, kk, vv)
    assert torch.equal(dx, again[0]) and torch.equal(dwq, again[1]) and torch.equal(dwk, again[2])


def test_empty_calls():
    e = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    w = e(64)
    q, k, v = attn_qk_norm_rope(e(2, 0, 4, 64), w, w, None, num_q_heads=2)
    assert q.shape == (2, 2, 0, 64)
    g = attn_qk_norm_rope_bwd(e(2, 0, 4, 64), w, w, None, q, k, v,
                              dq_weight=torch.ones(64, device="cuda"))
    assert not g[1].any() and not g[2].any()
    kp = e(1, 1, 64, 64)
    q = attn_qk_norm_rope_paged(e(0, 4, 64), w, w, None, i32([]), i32([]).long(), kp, kp.clone())
    o, lse = attn_decode_tree(q, kp, kp, i32([[0]]), i32([5]), i32([0, 0]), max_nodes=4)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    assert device_status() == 0
