"""The operators around the attention kernels, on the CPU: their plain definitions held to
worked examples, closed forms and differences, and the refusals of the binding and the C ABI."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle
from io_aware_softmax_b200 import _lib, api, build
from tests.test_binding_cpu import FakeLib, only_call, z

BF16, F32, U8, I32, I64 = (torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64)


# ------------------------------------------------------------------- the definitions

def test_page_tables_worked_example():
    # page size 4, a table of 3 pages a sequence; sequence 0 holds 3 rows in page 7 and adds 3,
    # sequence 1 adds nothing, sequence 2 begins with 5 and sequence 3 is full
    slots, pos, lens, off, used, table = oracle.page_tables(
        [3, 4, 0, 12], [3, 0, 5, 2], [20, 21, 22], [[7, 0, 0], [8, 0, 0], [0, 0, 0], [1, 2, 3]],
        page_size=4, num_tokens=12)
    assert off.tolist() == [0, 3, 3, 8, 10] and lens.tolist() == [6, 4, 5, 12]
    assert table.tolist() == [[7, 20, 0], [8, 0, 0], [21, 22, 0], [1, 2, 3]]
    assert slots.tolist() == [31, 80, 81, 84, 85, 86, 87, 88, -1, -1, -1, -1]
    assert pos.tolist() == [3, 4, 5, 0, 1, 2, 3, 4, 12, 13, 0, 0]
    assert used.tolist() == [3]


def test_page_tables_pool_runs_out_and_tokens_past_the_capacity_have_no_place():
    slots, pos, lens, off, used, table = oracle.page_tables(
        [0, 0], [6, 6], [5], [[9, 9, 9], [9, 9, 9]], page_size=2, num_tokens=8, free_used=0)
    assert table.tolist() == [[5, -1, -1], [-1, 9, 9]]
    assert slots.tolist() == [10, 11, -1, -1, -1, -1, -1, -1]
    assert off.tolist() == [0, 6, 8] and lens.tolist() == [6, 2] and used.tolist() == [4]


def test_page_tables_keeps_the_pages_of_rejected_rows():
    # 6 rows, then 4 drafted of which none was accepted: the second page is there already
    args = dict(page_size=4, num_tokens=5)
    _, _, lens, _, used, table = oracle.page_tables([3], [5], [7, 8], [[6, 0, 0]], **args)
    assert table.tolist() == [[6, 7, 0]] and lens.tolist() == [8] and used.tolist() == [1]
    slots, _, _, _, used, table = oracle.page_tables([3], [5], [7, 8], table, free_used=1,
                                                     held_rows=lens, **args)
    assert table.tolist() == [[6, 7, 0]] and used.tolist() == [1]
    assert slots.tolist() == [27, 28, 29, 30, 31]
    # more than the table has, or less than the rows
    assert oracle.page_tables([3], [5], [9], table, held_rows=[99], **args)[4].tolist() == [0]
    none = oracle.page_tables([3], [5], [9], table, held_rows=[-1], **args)
    assert none[5].tolist() == [[6, 9, 0]]


def test_tree_depth_and_bad_parents():
    parents = [-1, 0, 0, 1, 9, 5, -7]        # 4: not an earlier node, 5: itself
    assert [oracle.tree_depth(parents, i) for i in range(7)] == [0, 1, 1, 2, 0, 0, 0]
    assert [oracle.tree_depth(None, i) for i in range(4)] == [0, 1, 2, 3]


def test_page_tables_positions_are_the_depths_of_the_trees():
    rng = np.random.default_rng(6)
    new = [40, 1, 0, 25]
    parents = [int(rng.integers(-2, i + 2)) for n in new for i in range(n)]
    _, pos, _, off, _, _ = oracle.page_tables([7] * 4, new, range(9), [[0] * 9] * 4, 8, 66,
                                              parents=parents)
    for b, n in enumerate(new):
        mine = parents[off[b]:off[b + 1]]
        assert pos[off[b]:off[b + 1]].tolist() == [7 + oracle.tree_depth(mine, i)
                                                   for i in range(n)]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_the_complex_product(interleaved):
    rng = np.random.default_rng(0)
    rot, d = 16, 64
    a = rng.normal(size=(5, rot // 2))
    table = np.concatenate([np.cos(a), np.sin(a)], 1)
    x = rng.normal(size=(3, 2, d))
    y = oracle.rotate(x, table, [4, 0, 2], interleaved)
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, 8), slice(8, 16))
    want = (x[..., lo] + 1j * x[..., hi]) * np.exp(1j * a[[4, 0, 2]])[:, None]
    assert np.allclose(y[..., lo] + 1j * y[..., hi], want, atol=1e-14)
    assert np.array_equal(y[..., rot:], x[..., rot:])
    assert np.allclose(oracle.rotate(y, table, [4, 0, 2], interleaved, back=True), x, atol=1e-14)
    # a position outside the table reads zeros
    assert not oracle.rotate(x, table, [5, -1, 7], interleaved)[..., :rot].any()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("with_norm", [False, True])
def test_gradients_against_differences(interleaved, with_norm):
    rng = np.random.default_rng(1)
    T, Hq, Hkv, d, rot, eps = 3, 2, 1, 64, 32, 1e-3
    a = rng.normal(size=(8, rot // 2))
    table = np.concatenate([np.cos(a), np.sin(a)], 1)
    x = rng.normal(size=(T, Hq + 2 * Hkv, d))
    w = [1 + 0.3 * rng.normal(size=d) for _ in "qk"] if with_norm else [None, None]
    pos = [5, 0, 7]
    g = [rng.normal(size=(T, h, d)) for h in (Hq, Hkv, Hkv)]

    def loss(x, wq, wk):
        out = oracle.qk_norm_rope(x, wq, wk, table, pos, Hq, eps, interleaved)
        return sum((o * gg).sum() for o, gg in zip(out, g))

    dx, dwq, dwk = oracle.qk_norm_rope_backward(x, *w, table, pos, *g, eps, interleaved)
    h = 1e-6
    for i in (0, 50, 200, 300, 500, 700):
        step = np.zeros(x.size)
        step[i] = h
        step = step.reshape(x.shape)
        diff = (loss(x + step, *w) - loss(x - step, *w)) / (2 * h)
        assert abs(diff - dx.reshape(-1)[i]) < 1e-6
    if with_norm:
        for i in (0, 17, 63):
            e = np.zeros(d)
            e[i] = h
            diff = (loss(x, w[0] + e, w[1]) - loss(x, w[0] - e, w[1])) / (2 * h)
            assert abs(diff - dwq[i]) < 1e-6
            diff = (loss(x, w[0], w[1] + e) - loss(x, w[0], w[1] - e)) / (2 * h)
            assert abs(diff - dwk[i]) < 1e-6


def test_tree_is_attention_on_the_rows_of_each_path():
    # every node alone, on the context and its path, through the pinned decode definition
    rng = np.random.default_rng(2)
    Hq, Hkv, d, ps = 4, 2, 64, 64
    kp, vp = rng.normal(size=(2, 6, Hkv, ps, d))
    table = np.array([[3, 0, 5], [1, 4, 2]])
    offsets, lens = [0, 4, 6], [100, 130]
    parents = [-1, 0, 0, 2, -1, 0]
    q = rng.normal(size=(6, Hq, d))
    O, lse, _ = oracle.decode_tree(q, kp, vp, table, lens, offsets, parents)
    paths = [[0], [0, 1], [0, 2], [0, 2, 3], [0], [0, 1]]
    for t, path in enumerate(paths):
        b = int(t >= 4)
        n, L = (4, 100) if b == 0 else (2, 130)
        K, V = (oracle.gather_paged(p, table[b], L) for p in (kp, vp))
        rows = list(range(L - n)) + [L - n + j for j in path]
        want, want_l = oracle.attention(q[t][None, :, None], K[None][:, :, rows],
                                        V[None][:, :, rows])
        assert np.allclose(O[t], want[0, :, 0], atol=1e-12)
        assert np.allclose(lse[t], want_l[0, :, 0], atol=1e-12)


def test_tree_chain_and_missing_rows():
    rng = np.random.default_rng(3)
    q = rng.normal(size=(5, 2, 64))
    kp, vp = rng.normal(size=(2, 1, 1, 64, 64))
    chain = oracle.decode_tree(q, kp, vp, [[0]], [20], [0, 5])
    named = oracle.decode_tree(q, kp, vp, [[0]], [20], [0, 5], [-1, 0, 1, 2, 3])
    assert np.array_equal(chain[0], named[0])
    # fewer rows than drafted tokens: the first nodes have none
    O, lse, _ = oracle.decode_tree(q, kp, vp, [[0]], [2], [0, 5], [-1, -1, -1, 0, 3])
    assert np.isneginf(lse[:3]).all() and not O[:3].any()
    assert np.allclose(O[3], vp[0, 0, 0])


# ------------------------------------------------------------------------ the binding

class ServeLib(FakeLib):
    def attn_decode_tree_workspace_bytes(self, *a):
        return 4096

    def attn_qk_norm_rope_bwd_workspace_bytes(self, d):
        return 592 * 2 * d * 4


@pytest.fixture
def lib(monkeypatch):
    import contextlib
    fake = ServeLib()
    monkeypatch.setattr(api._lib, "load", lambda *a, **k: fake)
    monkeypatch.setattr(api, "_on_gpu", lambda t, name: None)
    monkeypatch.setattr(api, "_device", lambda t: contextlib.nullcontext())
    monkeypatch.setattr(api, "_stream", lambda device, stream=None: 0)
    monkeypatch.setattr(api, "_index", lambda t: 0)
    return fake


def test_calls_go_through_with_the_sizes(lib):
    out = api.attn_page_tables(z((3,), I32), z((3,), I32), z((9,), I32), z((3, 7), I32),
                               page_size=64, num_tokens=11, parents=z((11,), I32),
                               free_used=z((1,), I32))
    assert [tuple(t.shape) for t in out] == [(11,), (11,), (3,), (4,), (1,)]
    assert only_call(lib, "attn_page_tables")[12:17] == (3, 7, 64, 9, 11)
    lib.calls.clear()
    q, k, v = api.attn_qk_norm_rope(z((2, 5, 8, 64)), z((64,)), z((64,)), z((5, 32), F32),
                                    num_q_heads=4)
    assert q.shape == (2, 4, 5, 64) and k.shape == v.shape == (2, 2, 5, 64)
    assert only_call(lib, "attn_qk_norm_rope")[8:15] == (2, 5, 4, 2, 64, 32, 5)
    lib.calls.clear()
    g, wq, wk = api.attn_qk_norm_rope_bwd(z((2, 5, 8, 64)), z((64,)), z((64,)), None, q, k, v)
    assert g.shape == (2, 5, 8, 64) and wq.shape == wk.shape == (64,) and wq.dtype == F32
    assert only_call(lib, "attn_qk_norm_rope_bwd")[11:18] == (2, 5, 4, 2, 64, 0, 0)
    lib.calls.clear()
    q = api.attn_qk_norm_rope_paged(z((9, 8, 64)), None, None, z((100, 64), F32), z((9,), I32),
                                    z((9,), I64), z((3, 2, 64, 64)), z((3, 2, 64, 64)))
    assert q.shape == (9, 4, 64)
    assert only_call(lib, "attn_qk_norm_rope_paged")[9:17] == (9, 4, 2, 64, 3, 64, 64, 100)
    lib.calls.clear()
    o, lse = api.attn_decode_tree(q, z((3, 2, 64, 64)), z((3, 2, 64, 64)), z((5, 7), I32),
                                  z((5,), I32), z((6,), I32), max_nodes=4)
    assert o.shape == q.shape and lse.shape == (9, 4)
    assert only_call(lib, "attn_decode_tree")[9:18] == (5, 9, 4, 2, 3, 64, 7, 4, 64)


@pytest.mark.parametrize("change", [
    dict(new_lens=z((2,), I32)), dict(new_lens=z((3,), I64)), dict(block_table=z((2, 7), I32)),
    dict(parents=z((10,), I32)), dict(free_used=z((2,), I32)), dict(held_rows=z((2,), I32)),
    dict(slots=z((11,), I32)),
    dict(positions=z((12,), I32)), dict(seq_lens=z((4,), I32)), dict(token_offsets=z((3,), I32)),
    dict(pages_used=z((), I32)), dict(num_tokens=-1), dict(ctx_lens=z((6,), I32)[::2]),
    dict(free_pages=z((9,), I32, device="meta"))])
def test_page_tables_refusals(lib, change):
    a = dict(ctx_lens=z((3,), I32), new_lens=z((3,), I32), free_pages=z((9,), I32),
             block_table=z((3, 7), I32), page_size=64, num_tokens=11) | change
    with pytest.raises((ValueError, TypeError)):
        api.attn_page_tables(a.pop("ctx_lens"), a.pop("new_lens"), a.pop("free_pages"),
                             a.pop("block_table"), **a)
    assert lib.calls == []


@pytest.mark.parametrize("change", [
    dict(qkv=z((2, 5, 8, 64), F32)), dict(qkv=z((2, 5, 16, 64))[:, :, ::2]),
    dict(q_weight=None), dict(k_weight=z((32,))), dict(q_weight=z((64,), F32)),
    dict(rope_table=z((5, 32))), dict(rope_table=z((5, 32), F32, device="meta")),
    dict(num_q_heads=0), dict(num_q_heads=8), dict(num_q_heads=3),
    dict(positions=z((5,), I32)), dict(positions=z((2, 5), I64)), dict(q=z((2, 5, 4, 64))),
    dict(v=z((2, 2, 5, 64), F32))])
def test_qk_norm_rope_refusals(lib, change):
    a = dict(qkv=z((2, 5, 8, 64)), q_weight=z((64,)), k_weight=z((64,)),
             rope_table=z((5, 32), F32), num_q_heads=4) | change
    with pytest.raises((ValueError, TypeError)):
        api.attn_qk_norm_rope(**a)
    assert lib.calls == []


@pytest.mark.parametrize("change", [
    dict(dq=z((2, 4, 6, 64))), dict(dk=z((2, 3, 5, 64))), dict(dv=z((2, 1, 5, 64))),
    dict(dqkv=z((2, 5, 8, 32))), dict(dq_weight=z((64,))), dict(workspace=z((10,), U8)[::2]),
    dict(q_weight=None, k_weight=None, dk_weight=z((64,), F32)),
    dict(dv=z((2, 2, 5, 64), device="meta"))])
def test_qk_norm_rope_bwd_refusals(lib, change):
    a = dict(qkv=z((2, 5, 8, 64)), q_weight=z((64,)), k_weight=z((64,)),
             rope_table=z((5, 32), F32), dq=z((2, 4, 5, 64)), dk=z((2, 2, 5, 64)),
             dv=z((2, 2, 5, 64))) | change
    with pytest.raises((ValueError, TypeError)):
        api.attn_qk_norm_rope_bwd(**a)
    assert lib.calls == []


def test_a_table_too_short_for_the_default_positions(lib):
    x, w, g = z((2, 5, 8, 64)), z((64,)), [z((2, h, 5, 64)) for h in (4, 2, 2)]
    short, pos = z((4, 32), F32), z((2, 5), I32)
    with pytest.raises(ValueError, match="4 rows"):
        api.attn_qk_norm_rope(x, w, w, short, num_q_heads=4)
    with pytest.raises(ValueError, match="4 rows"):
        api.attn_qk_norm_rope_bwd(x, w, w, short, *g)
    assert lib.calls == []
    # positions that the host does not see, a table without angles, and nothing to rotate
    api.attn_qk_norm_rope(x, w, w, short, num_q_heads=4, positions=pos)
    api.attn_qk_norm_rope_bwd(x, w, w, short, *g, positions=pos)
    api.attn_qk_norm_rope(x, w, w, z((0, 0), F32), num_q_heads=4)
    api.attn_qk_norm_rope(x[:0], w, w, short, num_q_heads=4)
    assert len(lib.calls) == 4


@pytest.mark.parametrize("change", [
    dict(positions=None), dict(positions=z((8,), I32)), dict(slots=z((9,), I32)),
    dict(slots=z((8,), I64)), dict(k_pages=z((3, 2, 64, 128))), dict(v_pages=z((4, 2, 64, 64))),
    dict(k_pages=z((3, 4, 64, 64)), v_pages=z((3, 4, 64, 64))), dict(q=z((9, 8, 64))),
    dict(qkv=z((2, 9, 8, 64))), dict(v_pages=z((3, 2, 64, 64), device="meta"))])
def test_qk_norm_rope_paged_refusals(lib, change):
    a = dict(qkv=z((9, 8, 64)), q_weight=z((64,)), k_weight=z((64,)), rope_table=None,
             positions=z((9,), I32), slots=z((9,), I64), k_pages=z((3, 2, 64, 64)),
             v_pages=z((3, 2, 64, 64))) | change
    with pytest.raises((ValueError, TypeError)):
        api.attn_qk_norm_rope_paged(**a)
    assert lib.calls == []


@pytest.mark.parametrize("change", [
    dict(q=z((9, 4, 64), F32)), dict(q=z((1, 9, 4, 64))), dict(k_pages=z((3, 2, 64, 128))),
    dict(v_pages=z((3, 2, 128, 64))), dict(block_table=z((4, 7), I32)),
    dict(seq_lens=z((5,), I64)), dict(token_offsets=z((5,), I32)), dict(parents=z((8,), I32)),
    dict(out=z((9, 4, 64), F32)), dict(lse=z((4, 9), F32)), dict(workspace=z((64,), U8)[::2]),
    dict(block_table=z((5, 7), I32, device="meta"))])
def test_decode_tree_refusals(lib, change):
    a = dict(q=z((9, 4, 64)), k_pages=z((3, 2, 64, 64)), v_pages=z((3, 2, 64, 64)),
             block_table=z((5, 7), I32), seq_lens=z((5,), I32), token_offsets=z((6,), I32),
             max_nodes=4) | change
    with pytest.raises((ValueError, TypeError)):
        api.attn_decode_tree(**a)
    assert lib.calls == []


def test_sizes_past_32_bits_are_refused(lib):
    # 2^32 + 64 cut to 32 bits would be 64, a size that the library takes
    big = 2 ** 32 + 64
    m = lambda shape, t=BF16: z(shape, t, device="meta")  # noqa: E731
    i = m((3,), I32)
    tables = lambda **k: api.attn_page_tables(  # noqa: E731
        i, i, *(dict(free=m((9,), I32), table=m((3, 7), I32)) | k).values(), page_size=64,
        num_tokens=5)
    pages = lambda n, ps: m((n, 2, ps, 64))  # noqa: E731
    tree = lambda k, nodes=4, P=7: api.attn_decode_tree(  # noqa: E731
        m((3, 4, 64)), k, k, m((3, P), I32), i, m((4,), I32), max_nodes=nodes)
    w = m((64,))
    g = [m((1, h, 5, 64)) for h in (4, 2, 2)]
    for call in (
            lambda: tables(free=m((big,), I32)), lambda: tables(table=m((3, big), I32)),
            lambda: api.attn_page_tables(i, i, i, m((3, 7), I32), page_size=big, num_tokens=5),
            lambda: api.attn_page_tables(i, i, i, m((3, 7), I32), page_size=64 - 2 ** 32,
                                         num_tokens=5),
            lambda: api.attn_page_tables(i, i, i, m((3, 7), I32), page_size=64, num_tokens=big),
            lambda: api.attn_qk_norm_rope(m((1, 5, 8, 64)), w, w, m((big, 64), F32),
                                          num_q_heads=4),
            lambda: api.attn_qk_norm_rope(m((1, 5, 8, big)), None, None, None, num_q_heads=4),
            lambda: api.attn_qk_norm_rope_bwd(m((1, 5, 8, 64)), w, w, m((big, 64), F32), *g),
            lambda: api.attn_qk_norm_rope_paged(m((3, 8, 64)), w, w, None, i, i.long(),
                                                pages(big, 64), pages(big, 64)),
            lambda: tree(pages(3, big)), lambda: tree(pages(big, 64)),
            lambda: tree(pages(3, 64), nodes=2 ** 32 + 4), lambda: tree(pages(3, 64), P=big)):
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            call()
    assert lib.calls == []


def test_a_stream_of_another_device_is_refused(lib):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 7

    x, w, i = z((5, 8, 64)), z((64,)), z((5,), I32)
    pages = z((3, 2, 64, 64))
    g = [z((1, h, 5, 64)) for h in (4, 2, 2)]
    for call in (
            lambda: api.attn_page_tables(i, i, i, z((5, 7), I32), page_size=64, num_tokens=5,
                                         stream=Stream()),
            lambda: api.attn_qk_norm_rope(x[None], w, w, None, num_q_heads=4, stream=Stream()),
            lambda: api.attn_qk_norm_rope_bwd(x[None], w, w, None, *g, stream=Stream()),
            lambda: api.attn_qk_norm_rope_paged(x, w, w, None, i, i.long(), pages, pages,
                                                stream=Stream()),
            lambda: api.attn_decode_tree(x, pages, pages, z((5, 7), I32), i, z((6,), I32),
                                         max_nodes=4, stream=Stream())):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()
    assert lib.calls == []


# ------------------------------------------------------------------------- the sources

def test_kernels_that_start_early_read_with_ordinary_loads():
    # a kernel launched while the one before it runs may not read what that one writes through
    # the read-only path, whose loads the compiler may also move above the wait
    early = [s for s in build.SOURCES
             if "griddepcontrol.wait" in open(os.path.join(build.CSRC, s)).read()]
    assert early == ["attn_tree.cu"]
    for s in early:
        text = open(os.path.join(build.CSRC, s)).read()
        assert "__ldg" not in text and "ld.global.nc" not in text, s


# -------------------------------------------------------------------------- the C ABI

@pytest.fixture(scope="module")
def clib():
    build.build()
    return _lib.load()


def at(k, off=0):
    return ctypes.c_void_p((k << 24) + off)


def call(fn, args, **change):
    return fn(*(args | change).values())


def test_page_tables_status(clib):
    a = dict(ctx=at(1), new=at(2), free=at(3), used=at(4), held=at(12), parents=None,
             table=at(5), slots=at(6), pos=at(7), lens=at(8), off=at(9), out=at(10), B=3, P=7,
             ps=64, nf=9, T=11, stream=None)
    f = clib.attn_page_tables
    for change in (dict(B=-1), dict(P=-1), dict(ps=0), dict(nf=-1), dict(T=-1), dict(ctx=None),
                   dict(new=None), dict(free=None), dict(table=None), dict(slots=None),
                   dict(lens=None), dict(off=None), dict(out=None),
                   # an output on an input, and two outputs on each other
                   dict(lens=at(1)), dict(out=at(4)), dict(slots=at(7)), dict(lens=at(12, -4)),
                   dict(off=at(8, 8))):
        assert call(f, a, **change) == -1, change
    assert call(f, a, B=16385) == -2
    assert call(f, a, P=1 << 20, ps=4096) == -2
    assert call(f, a, slots=at(6, 8)) == -3
    assert call(f, a, pos=at(7, 4)) == -3
    assert call(f, a, parents=at(11, 2)) == -3


def test_qk_norm_rope_status(clib):
    a = dict(qkv=at(1), wq=at(2), wk=at(3), table=at(4), pos=None, q=at(5), k=at(6), v=at(7), B=2,
             N=5, Hq=4, Hkv=2, d=64, rot=32, rows=5, eps=1e-6, inter=0, stream=None)
    f = clib.attn_qk_norm_rope
    for change in (dict(B=-1), dict(N=-1), dict(Hq=-1), dict(Hkv=-1), dict(rot=-16), dict(rows=-1),
                   dict(wq=None), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")),
                   dict(qkv=None), dict(table=None), dict(q=None), dict(v=None)):
        assert call(f, a, **change) == -1, change
    for change in (dict(d=96), dict(rot=8), dict(rot=80), dict(N=1 << 30), dict(Hq=4093)):
        assert call(f, a, **change) == -2, change
    # an output on the input, on another output, on the angles
    for change in (dict(q=a["qkv"]), dict(v=at(6, 2 * 5 * 2 * 128 - 16)), dict(k=at(4, 16))):
        assert call(f, a, **change) == -1, change
    assert call(f, a, eps=1e-40) == -1
    for n in ("qkv", "wq", "wk", "table", "q", "k", "v"):
        assert call(f, a, **{n: at(20, 8)}) == -3, n
    assert call(f, a, pos=at(30, 2)) == -3
    assert call(f, a, B=0) == 0 and call(f, a, N=0) == 0 and call(f, a, Hq=0, Hkv=0) == 0


def test_a_table_too_short_for_the_default_positions_status(clib):
    a = dict(qkv=at(1), wq=at(2), wk=at(3), table=at(4), pos=None, q=at(5), k=at(6), v=at(7), B=2,
             N=5, Hq=4, Hkv=2, d=64, rot=32, rows=4, eps=1e-6, inter=0, stream=None)
    f = clib.attn_qk_norm_rope
    assert call(f, a) == -1 and call(f, a, rows=0) == -1 and call(f, a, table=None, rows=0) == -1
    assert call(f, a, B=0) == 0
    b = dict(qkv=at(1), wq=at(2), wk=at(3), table=at(4), pos=None, dq=at(5), dk=at(6), dv=at(7),
             dqkv=at(8), dwq=at(9), dwk=at(10), B=2, N=5, Hq=4, Hkv=2, d=64, rot=32, rows=4,
             eps=1e-6, inter=0, ws=at(11), bytes=1 << 20, stream=None)
    assert call(clib.attn_qk_norm_rope_bwd, b) == -1


def test_qk_norm_rope_paged_status(clib):
    a = dict(qkv=at(1), wq=at(2), wk=at(3), table=at(4), pos=at(8), slots=at(9), q=at(5), k=at(6),
             v=at(7), T=5, Hq=4, Hkv=2, d=64, pages=3, ps=64, rot=32, rows=5, eps=1e-6, inter=0,
             stream=None)
    f = clib.attn_qk_norm_rope_paged
    for change in (dict(T=-1), dict(pages=-1), dict(ps=0), dict(pos=None), dict(slots=None),
                   dict(q=None), dict(k=None), dict(wk=None)):
        assert call(f, a, **change) == -1, change
    assert call(f, a, v=a["k"]) == -1 and call(f, a, q=at(1, 256)) == -1
    assert call(f, a, d=32) == -2 and call(f, a, pages=1 << 20, ps=4096) == -2
    assert call(f, a, slots=at(9, 4)) == -3
    assert call(f, a, k=at(6, 8)) == -3
    assert call(f, a, T=0) == 0


def test_qk_norm_rope_bwd_status(clib):
    a = dict(qkv=at(1), wq=at(2), wk=at(3), table=at(4), pos=None, dq=at(5), dk=at(6), dv=at(7),
             dqkv=at(8), dwq=at(9), dwk=at(10), B=2, N=5, Hq=4, Hkv=2, d=64, rot=32, rows=5,
             eps=1e-6, inter=0, ws=at(11), bytes=1 << 20, stream=None)
    f = clib.attn_qk_norm_rope_bwd
    for change in (dict(dq=None), dict(dv=None), dict(dqkv=None), dict(dwq=None), dict(dwk=None),
                   dict(eps=-1.0), dict(B=-1)):
        assert call(f, a, **change) == -1, change
    need = clib.attn_qk_norm_rope_bwd_workspace_bytes(64)
    assert need == 592 * 2 * 64 * 4 and clib.attn_qk_norm_rope_bwd_workspace_bytes(0) == 0
    assert call(f, a, bytes=need - 1) == -6 and call(f, a, ws=None) == -6
    assert call(f, a, dqkv=a["qkv"]) == -1 and call(f, a, ws=at(8)) == -1
    assert call(f, a, dwq=at(30, 2)) == -3
    assert call(f, a, ws=at(11, 8)) == -3
    assert call(f, a, wq=None, wk=None, B=0) == 0


def test_decode_tree_status(clib):
    a = dict(q=at(1), k=at(2), v=at(3), table=at(4), lens=at(5), off=at(6), parents=None, o=at(7),
             lse=at(8), B=5, T=9, Hq=4, Hkv=2, pages=3, ps=64, P=7, nodes=4, d=64, scale=0.0,
             ws=at(9), bytes=1 << 28, stream=None)
    f = clib.attn_decode_tree
    for change in (dict(B=-1), dict(T=-1), dict(Hkv=0), dict(pages=-1), dict(ps=0), dict(P=-1),
                   dict(nodes=-1), dict(scale=float("nan")), dict(q=None), dict(k=None),
                   dict(table=None), dict(lens=None), dict(off=None), dict(o=None),
                   dict(lse=None)):
        assert call(f, a, **change) == -1, change
    for change in (dict(d=96), dict(ps=48), dict(nodes=129), dict(Hq=5), dict(Hq=34),
                   dict(P=1 << 20, ps=4096), dict(pages=1 << 30), dict(T=1 << 30)):
        assert call(f, a, **change) == -2, change
    for n in ("q", "k", "v", "o", "lse", "ws"):
        assert call(f, a, **{n: at(20, 8)}) == -3, n
    assert call(f, a, off=at(6, 2)) == -3
    need = clib.attn_decode_tree_workspace_bytes(5, 4, 2, 4, 64, 0)
    assert need > 0 and clib.attn_decode_tree_workspace_bytes(0, 4, 2, 4, 64, 0) == 0
    assert call(f, a, bytes=need - 1) == -6 and call(f, a, ws=None) == -6
    assert call(f, a, o=a["q"]) == -1 and call(f, a, lse=at(9, need - 16)) == -1
    assert call(f, a, T=0) == 0 and call(f, a, B=0) == 0 and call(f, a, nodes=0) == 0


def test_decode_tree_work_past_32_bits_a_cta(clib):
    # 40000 sequences of up to 2^30 rows: 2^24 units each, 2^39 in all
    a = dict(q=at(1), k=at(2), v=at(3), table=at(4), lens=at(5), off=at(6), parents=None, o=at(7),
             lse=at(8), B=40000, T=40000, Hq=4, Hkv=2, pages=3, ps=1 << 20, P=1 << 10, nodes=4,
             d=64, scale=0.0, ws=at(9), bytes=1 << 28, stream=None)
    assert call(clib.attn_decode_tree, a) == -2
    # few of them with tokens
    assert call(clib.attn_decode_tree, a, T=9, ws=None) == -6
