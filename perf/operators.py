"""The serving and training operators around the attention kernels, as they are measured.

Page tables and slots from request lengths; per-head norms of queries and keys with the rotary
rotation (forward, backward, and the form that writes the paged cache); attention of drafted
trees of tokens over a paged cache.  ``own`` selects between the plain torch forms and the
library's calls; both take what ``prepare`` gives.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6


def listed():
    return [
        # one step's bookkeeping of 64 decoding sequences, each adding one token
        dict(name="tables_decode", op="tables", B=64, max_pages=512, page=64, ctx=32000, new=1,
             tree=False, spare=0, mix=1),
        # a batch of drafted trees: a ragged number of nodes, positions by depth
        dict(name="tables_tree", op="tables", B=37, max_pages=300, page=128, ctx=16384, new=60,
             tree=True, spare=17, mix=2),
        # packed prompts of a large prefill step, the pages of every prompt new
        dict(name="tables_prefill", op="tables", B=256, max_pages=512, page=64, ctx=0, new=8192,
             tree=False, spare=1000, mix=3),
        # in front of causal training attention, one KV head for each query head
        dict(name="prep_mha", op="prep", B=8, N=4096, Hq=32, Hkv=32, d=128, rot=128,
             interleaved=False, far=False, norm=True),
        # its backward for grouped heads
        dict(name="prep_bwd_gqa", op="prep_bwd", B=4, N=4096, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, far=False, norm=True),
        # a small model's backward: odd length, half the head rotated, neighbouring pairs,
        # positions given
        dict(name="prep_bwd_small", op="prep_bwd", B=3, N=333, Hq=6, Hkv=2, d=64, rot=32,
             interleaved=True, far=True, norm=True),
        # one decode step: 16 tokens into a paged cache
        dict(name="paged_prep_decode", op="prep_paged", T=16, Hq=32, Hkv=8, d=128, rot=128,
             page=64, interleaved=False, norm=True),
        # a chunk of packed prompts into a paged cache
        dict(name="paged_prep_chunk", op="prep_paged", T=8191, Hq=32, Hkv=8, d=128, rot=128,
             page=64, interleaved=False, norm=True),
        # one user, a short text, a small tree
        dict(name="tree_one_short", op="tree", B=1, Hq=8, Hkv=2, d=64, page=64, ctx=1000,
             nodes=8, chain=False, mix=1),
        # a serving batch over long caches, trees of up to 16 nodes
        dict(name="tree_serving", op="tree", B=16, Hq=32, Hkv=8, d=128, page=64, ctx=32768,
             nodes=16, chain=False, mix=2),
        # wide trees: 64 nodes of 4 query heads share a KV head
        dict(name="tree_wide", op="tree", B=8, Hq=32, Hkv=8, d=128, page=128, ctx=8192,
             nodes=64, chain=False, mix=3),
        # a drafted line of up to 5 tokens, a KV head for each query head
        dict(name="tree_chain_mha", op="tree", B=7, Hq=16, Hkv=16, d=128, page=64, ctx=5000,
             nodes=5, chain=True, mix=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "prep", "prep_bwd", "prep_paged", "tree", "tree"])
    if op == "tables":
        page = rng.choice([16, 32, 64, 128])
        tree = rng.random() < 0.4
        new = _log(rng, 2, 96) if tree else _log(rng, 1, 8192)
        return dict(op=op, B=_log(rng, 1, 256), max_pages=-(-(32768 + 8192) // page), page=page,
                    ctx=rng.choice([0, _log(rng, 10, 32768)]), new=new, tree=tree,
                    spare=rng.randrange(100), mix=rng.randrange(1 << 20))
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    if op in ("prep", "prep_bwd"):
        Hq = Hkv * rng.choice([1, 2, 4, 5] if Hkv < 16 else [1, 2])
        most = 8 * 4096 * 96 * 128 if op == "prep" else 4 * 4096 * 48 * 128
        B = rng.randint(1, 8)
        N = _log(rng, 1, max(2, min(16384, most // (B * (Hq + 2 * Hkv) * d))))
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d // 2, 16, 0]),
                    interleaved=rng.random() < 0.4, far=rng.random() < 0.5,
                    norm=rng.random() < 0.8)
    if op == "prep_paged":
        Hq = Hkv * rng.choice([1, 2, 4, 7] if Hkv < 16 else [1, 2])
        return dict(op=op, T=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, d=d,
                    rot=rng.choice([d, d // 2, 16]), page=rng.choice([64, 128, 192]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.8)
    g = rng.choice([1, 2, 3, 4, 7, 8, 16] if Hkv <= 4 else [1, 2, 4, 5] if Hkv <= 8 else [1, 2])
    ctx = _log(rng, 100, 32768)
    most = 16 * 8 * 32768 * 128
    nodes = _log(rng, 1, min(96, 512 // g))
    B = min(_log(rng, 1, 64), max(1, most // (Hkv * (ctx + 256) * d * max(1, nodes * g // 64))))
    return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, d=d, page=rng.choice([64, 128, 192, 256]),
                ctx=ctx, nodes=nodes, chain=rng.random() < 0.3, mix=rng.randrange(1 << 20))


# ------------------------------------------------------------------------------- inputs

def _lengths(case):
    """Rows cached before the step, new tokens, and tree parents of every sequence: they go by
    the case alone, so that the sizes of the outputs do."""
    r = random.Random(case["mix"])
    B, most, new = case["B"], case["ctx"], case.get("nodes", case.get("new"))
    ctx = [r.randint((most + 1) // 2, most) for _ in range(B)]
    n = [r.randint((new + 3) // 4, new) for _ in range(B)]
    if B > 4:
        ctx[B // 2] = 0                 # a sequence that only begins
    parents = []
    for m in n:
        # a node hangs on one of the 6 before it, or on the context
        parents += [max(-1, i - 1 - r.randrange(6)) for i in range(m)]
    return ctx, n, parents


def _total(case):
    return sum(_lengths(case)[1])


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", dtype=torch.bfloat16, generator=g)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _rope_table(rows, rot):
    """cos | sin of pos * 10000^(-2 i / rot), the angles in 64 bits."""
    if rot == 0:
        return None
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _weights(g, case):
    if not case["norm"]:
        return None, None
    d = case["d"]
    return tuple((1 + 0.2 * torch.randn(d, device="cuda", generator=g)).bfloat16() for _ in "qk")


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "tables":
        ctx, n, parents = _lengths(case)
        B, ps, P = case["B"], case["page"], case["max_pages"]
        T = sum(n) + case["spare"]
        have = [-(-c // ps) for c in ctx]
        need = [-(-(c + m) // ps) - h for c, m, h in zip(ctx, n, have)]
        pages = torch.randperm(sum(have) + sum(need) + 64, device="cuda", generator=g).int()
        table = torch.full((B, P), -1, dtype=torch.int32, device="cuda")
        first = np.cumsum([0] + have)
        held = torch.arange(P, device="cuda")[None, :]
        at = _ints(first[:-1].tolist())[:, None] + held
        table = torch.where(held < _ints(have)[:, None], pages[at.clamp(max=len(pages) - 1)], table)
        return dict(case=case, ctx=_ints(ctx), new=_ints(n), free=pages[sum(have):].contiguous(),
                    table=table.contiguous(), T=T,
                    parents=_ints(parents + [-1] * case["spare"]) if case["tree"] else None)
    if op in ("prep", "prep_bwd"):
        B, N, Hq, Hkv, d = (case[k] for k in ("B", "N", "Hq", "Hkv", "d"))
        wq, wk = _weights(g, case)
        s = dict(case=case, qkv=_randn(g, B, N, Hq + 2 * Hkv, d), wq=wq, wk=wk, positions=None)
        rows = N
        if case["far"]:
            rows = 131072
            s["positions"] = torch.randint(0, rows - N, (B, 1), device="cuda", generator=g).int() \
                + torch.arange(N, device="cuda", dtype=torch.int32)
        s["table"] = _rope_table(rows, case["rot"])
        if op == "prep_bwd":
            s["dq"], s["dk"], s["dv"] = (_randn(g, B, h, N, d) for h in (Hq, Hkv, Hkv))
        return s
    if op == "prep_paged":
        T, Hq, Hkv, d, ps = (case[k] for k in ("T", "Hq", "Hkv", "d", "page"))
        wq, wk = _weights(g, case)
        pages = -(-T // ps) + 16
        slots = torch.randperm(pages * ps, device="cuda", generator=g)[:T].contiguous()
        if T > 1:
            slots[T // 2] = -1          # a token without a place in the cache
        return dict(case=case, qkv=_randn(g, T, Hq + 2 * Hkv, d), wq=wq, wk=wk, slots=slots,
                    positions=torch.randint(0, 32768, (T,), device="cuda", generator=g).int(),
                    table=_rope_table(32768, case["rot"]), k=_randn(g, pages, Hkv, ps, d),
                    v=_randn(g, pages, Hkv, ps, d))
    ctx, n, parents = _lengths(case)
    B, Hq, Hkv, d, ps = (case[k] for k in ("B", "Hq", "Hkv", "d", "page"))
    held = [-(-(c + m) // ps) for c, m in zip(ctx, n)]
    P = max(held)
    order = torch.randperm(sum(held), device="cuda", generator=g).int()
    at = _ints(np.cumsum([0] + held)[:-1].tolist())[:, None] + torch.arange(P, device="cuda")
    table = torch.where(torch.arange(P, device="cuda")[None, :] < _ints(held)[:, None],
                        order[at.clamp(max=sum(held) - 1)], 0).int().contiguous()
    return dict(case=case, q=_randn(g, sum(n), Hq, d), k=_randn(g, sum(held), Hkv, ps, d),
                v=_randn(g, sum(held), Hkv, ps, d), table=table,
                lens=_ints([c + m for c, m in zip(ctx, n)]),
                offsets=_ints(np.cumsum([0] + n).tolist()),
                parents=None if case["chain"] else _ints(parents))


# -------------------------------------------------------------------------- plain forms

def _plain_tables(s):
    case, T = s["case"], s["T"]
    ps, P = case["page"], case["max_pages"]
    cap = P * ps
    c = s["ctx"].long().clamp(0, cap)
    off = torch.cat([c.new_zeros(1), s["new"].long().clamp(min=0).cumsum(0)]).clamp(max=T)
    e = (c + off[1:] - off[:-1]).clamp(max=cap)
    have = (c + ps - 1) // ps
    need = (e + ps - 1) // ps - have
    first = need.cumsum(0) - need
    col = torch.arange(P, device=c.device)[None, :]
    x = first[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    free = s["free"]
    page = torch.where(x < len(free), free[x.clamp(0, len(free) - 1)], -1)
    s["table"].copy_(torch.where(fresh, page, s["table"]))
    t = torch.arange(T, device=c.device)
    b = torch.searchsorted(off[1:].contiguous(), t, right=True).clamp(max=case["B"] - 1)
    real = t < off[-1]
    i = t - off[b]
    row = c[b] + i
    pg = s["table"][b, (row // ps).clamp(max=P - 1)].long()
    slots = torch.where(real & (row < cap) & (pg >= 0), pg * ps + row % ps, -1)
    pos = row
    if s["parents"] is not None:
        p = s["parents"].long()
        p = torch.where((p >= 0) & (p < i), p, -1)
        up = torch.where(p >= 0, off[b] + p, T)             # T: the context
        depth = torch.cat([(p >= 0).long(), p.new_zeros(1)])
        up = torch.cat([up, up.new_full((1,), T)])
        for _ in range(max(1, T.bit_length())):
            depth = depth + depth[up]
            up = up[up]
        pos = c[b] + depth[:-1]
    pos = torch.where(real, pos, 0)
    used = need.sum()
    return (slots, pos.int(), e.int(), off.int(), used.reshape(1).int(), s["table"])


def _rotate(x, table, pos, rot, interleaved, sign):
    """x [.., tokens, heads, d] fp32, pos [.., tokens]."""
    if rot == 0:
        return x
    cs = table[pos.long()][..., None, :]
    cos, sin = cs[..., : rot // 2], cs[..., rot // 2:] * sign
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _positions(s):
    if s["positions"] is not None:
        return s["positions"]
    B, N = s["qkv"].shape[:2]
    return torch.arange(N, device="cuda").expand(B, N)


def _normed(x, w):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _plain_prep(s):
    c = s["case"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    x = s["qkv"].float()
    q, k, v = x.split([Hq, Hkv, Hkv], -2)
    pos = _positions(s)
    q = _rotate(_normed(q, s["wq"]), s["table"], pos, c["rot"], c["interleaved"], 1)
    k = _rotate(_normed(k, s["wk"]), s["table"], pos, c["rot"], c["interleaved"], 1)
    return q, k, v


def _plain_prep_train(s):
    return tuple(t.transpose(1, 2).bfloat16().contiguous() for t in _plain_prep(s))


def _plain_norm_bwd(x, w, dz):
    if w is None:
        return dz, None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    dxn = dz * w.float()
    dx = r * dxn - x * (r * r * r) * (x * dxn).mean(-1, keepdim=True)
    return dx, (dz * x * r).sum((0, 1, 2), dtype=torch.float64).float()


def _plain_prep_bwd(s):
    c = s["case"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    x = s["qkv"].float()
    pos = _positions(s)
    out = []
    for xs, w, dy in ((x[..., :Hq, :], s["wq"], s["dq"]), (x[..., Hq:Hq + Hkv, :], s["wk"], s["dk"])):
        dz = _rotate(dy.float().transpose(1, 2), s["table"], pos, c["rot"], c["interleaved"], -1)
        out.append(_plain_norm_bwd(xs, w, dz))
    (dq, dwq), (dk, dwk) = out
    dqkv = torch.cat([dq, dk, s["dv"].float().transpose(1, 2)], 2).bfloat16()
    return (dqkv, dwq, dwk) if dwq is not None else (dqkv,)


def _plain_prep_paged(s):
    q, k, v = _plain_prep(s)
    ps = s["case"]["page"]
    keep = s["slots"] >= 0
    # a token without a slot puts the same as the first token that has one
    t = torch.where(keep, torch.arange(len(keep), device="cuda"), keep.int().argmax())
    sl = s["slots"][t]
    for pages, x in ((s["k"], k), (s["v"], v)):
        pages[sl // ps, :, sl % ps] = x[t].bfloat16()
    return q.bfloat16(), s["k"], s["v"]


def _plain_tree(s):
    c = s["case"]
    Hq, Hkv, d, n = c["Hq"], c["Hkv"], c["d"], c["nodes"]
    B, P = s["table"].shape
    off = s["offsets"].long()
    cnt = off[1:] - off[:-1]
    T = s["q"].shape[0]
    node = torch.arange(n, device="cuda")
    at = (off[:-1, None] + node).clamp(max=T - 1)                       # [B, n]
    q = s["q"][at].float().transpose(1, 2).reshape(B, Hkv, Hq // Hkv, n, d)
    k = s["k"][s["table"].long()].transpose(1, 2).reshape(B, Hkv, 1, -1, d).float()
    v = s["v"][s["table"].long()].transpose(1, 2).reshape(B, Hkv, 1, -1, d).float()
    if s["parents"] is None:
        sees = (node[None, :] <= node[:, None]).expand(B, n, n)
    else:
        p = torch.where(node < cnt[:, None], s["parents"][at].long(), -1)
        sees = (node[None, None, :] == p[:, :, None]) | torch.eye(n, dtype=torch.bool, device="cuda")
        for _ in range(max(1, n.bit_length())):
            sees = (sees.float() @ sees.float()) > 0
    L = s["lens"].long()[:, None, None]
    key = torch.arange(k.shape[3], device="cuda")[None, None, :]
    j = key - (L - cnt[:, None, None])                                  # [B, 1, keys]
    tree = torch.gather(sees, 2, j.clamp(0, n - 1).expand(B, n, -1))
    see = ((j < 0) | tree) & (key < L)
    x = (q.reshape(B, Hkv, -1, d) * (1 / math.sqrt(d))) @ k[:, :, 0].transpose(-1, -2)
    x = x.reshape(B, Hkv, Hq // Hkv, n, -1).masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x.reshape(B, Hkv, -1, x.shape[-1]) @ v[:, :, 0]).reshape(B, Hkv, -1, n, d) / l
    lse = (m + l.log())[..., 0]
    b = torch.searchsorted(off[1:].contiguous(), torch.arange(T, device="cuda"), right=True)
    i = torch.arange(T, device="cuda") - off[b]
    o = o.reshape(B, Hq, n, d)[b, :, i].bfloat16()
    return o, lse.reshape(B, Hq, n)[b, :, i].contiguous()


# ------------------------------------------------------------------------------ one pass

def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if not own:
        return {"tables": _plain_tables, "prep": _plain_prep_train, "prep_bwd": _plain_prep_bwd,
                "prep_paged": _plain_prep_paged, "tree": _plain_tree}[op](s)
    import io_aware_softmax_b200 as attn
    if op == "tables":
        slots, pos, lens, off, used = attn.attn_page_tables(
            s["ctx"], s["new"], s["free"], s["table"], page_size=c["page"], num_tokens=s["T"],
            parents=s["parents"])
        return slots, pos, lens, off, used, s["table"]
    if op == "prep":
        return attn.attn_qk_norm_rope(s["qkv"], s["wq"], s["wk"], s["table"], num_q_heads=c["Hq"],
                                      positions=s["positions"], eps=EPS,
                                      interleaved=c["interleaved"])
    if op == "prep_bwd":
        out = attn.attn_qk_norm_rope_bwd(s["qkv"], s["wq"], s["wk"], s["table"], s["dq"], s["dk"],
                                         s["dv"], positions=s["positions"], eps=EPS,
                                         interleaved=c["interleaved"])
        return out if c["norm"] else out[:1]
    if op == "prep_paged":
        q = attn.attn_qk_norm_rope_paged(s["qkv"], s["wq"], s["wk"], s["table"], s["positions"],
                                         s["slots"], s["k"], s["v"], eps=EPS,
                                         interleaved=c["interleaved"])
        return q, s["k"], s["v"]
    return attn.attn_decode_tree(s["q"], s["k"], s["v"], s["table"], s["lens"], s["offsets"],
                                 max_nodes=c["nodes"], parents=s["parents"])


def work(case):
    op = case["op"]
    if op == "tables":
        ctx, n, _ = _lengths(case)
        ps, B, T = case["page"], case["B"], sum(n) + case["spare"]
        have = [-(-c // ps) for c in ctx]
        new_pages = sum(-(-(c + m) // ps) - h for c, m, h in zip(ctx, n, have))
        # lengths in and out, offsets, the new pages from the pool to the table, the last held
        # page of each sequence, 8 + 4 bytes a token (and its parent)
        return {"bytes": 16 * B + 8 * new_pages + 4 * B + T * (16 if case["tree"] else 12),
                "flops": 0}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if op == "tree":
        ctx, n, _ = _lengths(case)
        rows = sum(c + m for c, m in zip(ctx, n))
        # the cached rows' K and V, q and o, lse
        return {"bytes": rows * Hkv * d * 4 + sum(n) * Hq * (4 * d + 4),
                "flops": 4 * d * Hq * sum(m * (c + m) for c, m in zip(ctx, n))}
    T = case["T"] if op == "prep_paged" else case["B"] * case["N"]
    heads = Hq + 2 * Hkv
    rows = min(T, 32768 if op == "prep_paged" or case["far"] else case["N"])
    bytes_ = 4 * T * heads * d + 4 * rows * case["rot"]
    if op == "prep_paged":
        bytes_ += 12 * T
    if op == "prep_bwd":
        bytes_ += 2 * T * (Hq + Hkv) * d * (1 if case["norm"] else 0)
    return {"bytes": bytes_, "flops": T * heads * d * (16 if op == "prep_bwd" else 8)}


# ------------------------------------------------------- the definitions, in 64 bits

def _exact_angles(s, shape):
    """cos and sin of every token in 64 bits (the table's own values: it is an input)."""
    rot = s["case"]["rot"]
    if s["positions"] is None:
        pos = torch.arange(shape[1], device="cuda").repeat(shape[0], 1)
    else:
        pos = s["positions"].long()
    t = s["table"].index_select(0, pos.reshape(-1)).double().reshape(*pos.shape, 1, rot)
    return t.chunk(2, -1)


def _exact_pairs(rot, interleaved):
    h = torch.arange(rot // 2, device="cuda")
    return (2 * h, 2 * h + 1) if interleaved else (h, h + rot // 2)


def _exact_rotated(s, z, back):
    c = s["case"]
    if c["rot"] == 0:
        return z
    cos, sin = _exact_angles(s, z.shape)
    lo, hi = _exact_pairs(c["rot"], c["interleaved"])
    y = z.clone()
    a, b = z[..., lo], z[..., hi]
    if back:
        y[..., lo] = cos * a + sin * b
        y[..., hi] = cos * b - sin * a
    else:
        y[..., lo] = cos * a - sin * b
        y[..., hi] = sin * a + cos * b
    return y


def _exact_heads(s, x, w):
    if w is None:
        return _exact_rotated(s, x, False)
    size = torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)
    return _exact_rotated(s, x / size * w.double(), False)


def _exact_prep(s):
    c = s["case"]
    x = s["qkv"].double()
    q = _exact_heads(s, x[..., : c["Hq"], :], s["wq"])
    k = _exact_heads(s, x[..., c["Hq"]: c["Hq"] + c["Hkv"], :], s["wk"])
    return q, k, x[..., c["Hq"] + c["Hkv"]:, :]


def _exact_prep_bwd(s):
    c = s["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    parts, gains = [], []
    for lo, hi, w, dy in ((0, Hq, s["wq"], s["dq"]), (Hq, Hq + Hkv, s["wk"], s["dk"])):
        x = s["qkv"][..., lo:hi, :].double()
        dz = _exact_rotated(s, dy.permute(0, 2, 1, 3).double(), True)
        if w is None:
            parts.append(dz)
            continue
        size = torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS)
        u = x / size
        gains.append(torch.einsum("bnhd,bnhd->d", dz, u))
        t = dz * w.double()
        parts.append((t - u * (u * t).sum(-1, keepdim=True) / d) / size)
    parts.append(s["dv"].permute(0, 2, 1, 3).double())
    return (torch.cat(parts, 2), *gains)


def _exact_prep_paged(s):
    q, k, v = _exact_prep(s)
    out = [q]
    slots = s["slots"].tolist()
    t = torch.tensor([i for i, x in enumerate(slots) if x >= 0], device="cuda", dtype=torch.long)
    to = torch.tensor([x for x in slots if x >= 0], device="cuda", dtype=torch.long)
    for pages, x in ((s["k"], k), (s["v"], v)):
        p, h, ps, d = pages.shape
        flat = pages.double().permute(0, 2, 1, 3).reshape(p * ps, h, d)
        flat[to] = x[t]
        out.append(flat.reshape(p, ps, h, d).permute(0, 2, 1, 3).contiguous())
    return tuple(out)


def _exact_tables(s):
    case = s["case"]
    ps, P, T = case["page"], case["max_pages"], s["T"]
    ctx, new, free = s["ctx"].tolist(), s["new"].tolist(), s["free"].tolist()
    table = s["table"].cpu().numpy().copy()
    parents = None if s["parents"] is None else s["parents"].tolist()
    slots, pos = np.full(T, -1, np.int64), np.zeros(T, np.int32)
    lens, off, used = [], [0], 0
    for b, (c, m) in enumerate(zip(ctx, new)):
        m = min(m, T - off[-1])
        e = min(c + m, P * ps)
        for p in range(-(-c // ps), -(-e // ps)):
            table[b, p] = free[used] if used < len(free) else -1
            used += 1
        rows = np.arange(c, e)
        pages = table[b, rows // ps].astype(np.int64)
        o = off[-1]
        slots[o:o + e - c] = np.where(pages >= 0, pages * ps + rows % ps, -1)
        depth = list(range(m))
        if parents is not None:
            for i in range(m):
                p = parents[o + i]
                depth[i] = depth[p] + 1 if 0 <= p < i else 0
        pos[o:o + m] = c + np.array(depth, np.int32)
        lens.append(e)
        off.append(o + m)
    return (torch.from_numpy(slots), torch.from_numpy(pos), _ints(lens), _ints(off), _ints([used]),
            torch.from_numpy(table))


def _exact_tree(s):
    c = s["case"]
    Hq, Hkv, d, ps = c["Hq"], c["Hkv"], c["d"], c["page"]
    g = Hq // Hkv
    off, lens = s["offsets"].tolist(), s["lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    parents = None if s["parents"] is None else s["parents"].tolist()
    for b, L in enumerate(lens):
        m = off[b + 1] - off[b]
        see = torch.zeros(m, L, dtype=torch.bool)
        see[:, : L - m] = True
        for i in range(m):
            j = i
            while j >= 0:
                see[i, L - m + j] = True
                j = j - 1 if parents is None else parents[off[b] + j]
        see = see.cuda()
        at = s["table"][b, : -(-L // ps)].long()
        for h in range(Hkv):
            k = s["k"][at, h].reshape(-1, d)[:L].double()
            v = s["v"][at, h].reshape(-1, d)[:L].double()
            q = s["q"][off[b]:off[b + 1], h * g:(h + 1) * g].double()
            x = torch.einsum("ihd,td->iht", q, k) / d ** 0.5
            x = torch.where(see[:, None], x, -torch.inf)
            out[off[b]:off[b + 1], h * g:(h + 1) * g] = torch.softmax(x, -1) @ v
            lse[off[b]:off[b + 1], h * g:(h + 1) * g] = torch.logsumexp(x, -1)
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tables":
        return _exact_tables(s)
    if op == "prep":
        return tuple(t.permute(0, 2, 1, 3).contiguous() for t in _exact_prep(s))
    if op == "prep_bwd":
        return _exact_prep_bwd(s)
    if op == "prep_paged":
        return _exact_prep_paged(s)
    return _exact_tree(s)
