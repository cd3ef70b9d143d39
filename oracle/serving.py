"""The plain definitions, in fp64 numpy, of the operators around the attention kernels: page
tables and slots, per-head norms with the rotary rotation and their gradients, and attention
of drafted trees over a paged cache."""
from __future__ import annotations

import numpy as np

from .attention import default_scale


def tree_parent(parents, i: int) -> int:
    """Node i's parent in one sequence's parents (None: a chain); an entry that is not an
    earlier node counts as -1."""
    if parents is None:
        return i - 1
    p = int(parents[i])
    return p if 0 <= p < i else -1


def tree_depth(parents, i: int) -> int:
    depth = 0
    while (i := tree_parent(parents, i)) >= 0:
        depth += 1
    return depth


def page_tables(ctx_lens, new_lens, free_pages, block_table, page_size: int, num_tokens: int,
                free_used: int = 0, parents=None, held_rows=None):
    """(slots, positions, seq_lens, token_offsets, pages_used, block_table) of one step."""
    table = np.array(block_table, dtype=np.int32)
    B, P = table.shape
    cap = P * page_size
    slots = np.full(num_tokens, -1, np.int64)
    positions = np.zeros(num_tokens, np.int32)
    offsets, seq_lens, used = [0], [], max(int(free_used), 0)
    for b in range(B):
        c = min(max(int(ctx_lens[b]), 0), cap)
        o = offsets[-1]
        n = min(max(int(new_lens[b]), 0), num_tokens - o)
        end = min(c + n, cap)
        owned = c if held_rows is None else min(max(int(held_rows[b]), c), cap)
        for p in range(-(-owned // page_size), -(-end // page_size)):
            table[b, p] = free_pages[used] if used < len(free_pages) else -1
            used += 1
        depths = list(range(n))
        if parents is not None:
            mine = parents[o:o + n]
            for i in range(n):              # a parent comes before its node
                p = tree_parent(mine, i)
                depths[i] = depths[p] + 1 if p >= 0 else 0
        for i in range(n):
            if c + i < cap and table[b, (c + i) // page_size] >= 0:
                slots[o + i] = int(table[b, (c + i) // page_size]) * page_size + (c + i) % page_size
            positions[o + i] = c + depths[i]
        seq_lens.append(end)
        offsets.append(o + n)
    return (slots, positions, np.array(seq_lens, np.int32), np.array(offsets, np.int32),
            np.array([used], np.int32), table)


def _pairs(rot: int, interleaved: bool):
    h = np.arange(rot // 2)
    return (2 * h, 2 * h + 1) if interleaved else (h, h + rot // 2)


def _angles(table, positions):
    """cos, sin [tokens, rot / 2]; a position outside the table has zeros for both."""
    table = np.asarray(table, np.float64)
    pos = np.asarray(positions).astype(np.int64)
    inside = (pos >= 0) & (pos < table.shape[0])
    row = np.zeros((len(pos), table.shape[1]))
    row[inside] = table[pos[inside]]
    return np.split(row, 2, axis=1)


def rotate(z, table, positions, interleaved: bool = False, back: bool = False):
    """z [tokens, heads, d] rotated by each token's angles (back: by the transpose)."""
    y = np.array(z, np.float64)
    if table is None or table.shape[1] == 0:
        return y
    cos, sin = (a[:, None, :] for a in _angles(table, positions))
    if back:
        sin = -sin
    lo, hi = _pairs(table.shape[1], interleaved)
    a, b = y[..., lo].copy(), y[..., hi].copy()
    y[..., lo] = a * cos - b * sin
    y[..., hi] = b * cos + a * sin
    return y


def norm(x, w, eps: float):
    x = np.asarray(x, np.float64)
    if w is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def qk_norm_rope(qkv, q_weight, k_weight, table, positions, num_q_heads: int, eps: float,
                 interleaved: bool = False):
    """qkv [tokens, H, d] -> (q, k, v), each [tokens, heads, d]."""
    qkv = np.asarray(qkv, np.float64)
    kv = (qkv.shape[1] - num_q_heads) // 2
    q = rotate(norm(qkv[:, :num_q_heads], q_weight, eps), table, positions, interleaved)
    k = rotate(norm(qkv[:, num_q_heads:num_q_heads + kv], k_weight, eps), table, positions,
               interleaved)
    return q, k, qkv[:, num_q_heads + kv:]


def norm_backward(x, w, dz, eps: float):
    """(dx, dw) of norm for the gradient dz of its result."""
    if w is None:
        return np.asarray(dz, np.float64), None
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    t = dz * w
    dx = r * t - x * r ** 3 * (x * t).mean(-1, keepdims=True)
    return dx, (dz * x * r).sum((0, 1))


def qk_norm_rope_backward(qkv, q_weight, k_weight, table, positions, dq, dk, dv, eps: float,
                          interleaved: bool = False):
    """(dqkv, dq_weight, dk_weight); dq, dk, dv [tokens, heads, d]."""
    qkv = np.asarray(qkv, np.float64)
    nq, nk = dq.shape[1], dk.shape[1]
    gq, wq = norm_backward(qkv[:, :nq], q_weight,
                           rotate(dq, table, positions, interleaved, back=True), eps)
    gk, wk = norm_backward(qkv[:, nq:nq + nk], k_weight,
                           rotate(dk, table, positions, interleaved, back=True), eps)
    return np.concatenate([gq, gk, np.asarray(dv, np.float64)], 1), wq, wk


def decode_tree(q, k_pages, v_pages, block_table, seq_lens, token_offsets, parents=None,
                scale=None, max_nodes: int = 128):
    """(O [T, Hq, d], LSE [T, Hq], A): the plain attention of every drafted node over the rows
    it sees, A = sum_j P_j |V_j| (what a rounding of P can move O by).  Rows that belong to no
    sequence, or lie past max_nodes, are NaN."""
    q, kp, vp = (np.asarray(x, np.float64) for x in (q, k_pages, v_pages))
    T, Hq, d = q.shape
    pages, Hkv, ps, _ = kp.shape
    cap = np.asarray(block_table).shape[1] * ps
    scale = scale if scale is not None and scale > 0 else default_scale(d)
    O, A = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse = np.full((T, Hq), np.nan)
    for b in range(len(seq_lens)):
        first, n = int(token_offsets[b]), int(token_offsets[b + 1]) - int(token_offsets[b])
        length = min(max(int(seq_lens[b]), 0), cap)
        row = np.arange(length)
        page = np.asarray(block_table)[b, row // ps] if length else row
        good = (page >= 0) & (page < pages)
        K, V = np.zeros((Hkv, length, d)), np.zeros((Hkv, length, d))
        K[:, good] = kp[page[good], :, row[good] % ps].transpose(1, 0, 2)
        V[:, good] = vp[page[good], :, row[good] % ps].transpose(1, 0, 2)
        mine = None if parents is None else parents[first:first + n]
        for i in range(min(n, max_nodes)):
            see = row < length - n
            j = i
            while j >= 0:
                if 0 <= length - n + j < length:
                    see[length - n + j] = True
                j = tree_parent(mine, j)
            for h in range(Hq):
                g = h // (Hq // Hkv)
                if not see.any():
                    O[first + i, h], A[first + i, h], lse[first + i, h] = 0, 0, -np.inf
                    continue
                s = K[g, see] @ q[first + i, h] * scale
                m = s.max()
                e = np.exp(s - m)
                O[first + i, h] = e @ V[g, see] / e.sum()
                A[first + i, h] = e @ np.abs(V[g, see]) / e.sum()
                lse[first + i, h] = m + np.log(e.sum())
    return O, lse, A
