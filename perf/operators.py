"""The serving step's operators around the paged cache, as cases to time.

Four operators of one serving loop, each with its plain form in torch:

  slots    the step's page tables, slots, positions and lengths from the
           requests' cached and new token counts (paged_kv_slots)
  write    the step's new K and V rows into the pages (paged_kv_write)
  tree     attention of each request's tree of drafted tokens over its cache
           (paged_gqa_tree)
  prefill  causal attention of whole packed prompts, before their K and V
           are in any cache (packed_gqa_prefill)

``own`` False: the plain forms (fp32, rounded once at the end).  ``own`` True:
the library's entry points.  Sizes follow from the case alone ("sizes" seeds
the drawn lengths); the values and the placement of pages follow from the
seed of ``prepare``.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small batch: launch latency
        dict(name="slots_step", op="slots", seqs=64, block=16, ctx=4096, new=1, prompts=0,
             prompt=0, spare=0, sizes=1),
        # a continuous-batching step: decode steps beside chunks of new prompts, in a
        # launch of a fixed row count (the rows behind the last request are padding)
        dict(name="slots_mixed", op="slots", seqs=257, block=16, ctx=8192, new=4, prompts=17,
             prompt=2048, spare=117, sizes=2),
        # admission of many prompts at once, short pages
        dict(name="slots_bulk", op="slots", seqs=2048, block=8, ctx=512, new=1, prompts=2000,
             prompt=511, spare=0, sizes=3),
        # the new token of each request of a decode batch
        dict(name="write_step", op="write", rows=64, q_heads=32, kv_heads=8, dim=128, block=16,
             layout="head_major", skip=0, sizes=1),
        # a step of mixed prompts in short pages of a token-major cache, padded rows among them
        dict(name="write_prompt", op="write", rows=10007, q_heads=24, kv_heads=4, dim=256,
             block=8, layout="token_major", skip=500, sizes=2),
        # a long admission: 131 k rows of new prompts
        dict(name="write_bulk", op="write", rows=131072, q_heads=32, kv_heads=8, dim=128,
             block=32, layout="head_major", skip=0, sizes=3),
        # one request verifying a small tree: latency
        dict(name="tree_one", op="tree", seqs=1, q_heads=32, kv_heads=8, dim=128, block=16,
             ctx_lo=1000, ctx_hi=1000, nodes_lo=8, nodes_hi=8, sizes=1),
        # a batch of requests with trees of different sizes
        dict(name="tree_batch", op="tree", seqs=64, q_heads=32, kv_heads=8, dim=128, block=16,
             ctx_lo=512, ctx_hi=4096, nodes_lo=5, nodes_hi=32, sizes=2),
        # long contexts at head_dim 256
        dict(name="tree_long", op="tree", seqs=32, q_heads=16, kv_heads=2, dim=256, block=32,
             ctx_lo=8192, ctx_hi=32768, nodes_lo=16, nodes_hi=24, sizes=3),
        # many short prompts of different lengths, from one token on
        dict(name="prefill_short", op="prefill", seqs=37, q_heads=24, kv_heads=4, dim=256,
             len_lo=1, len_hi=512, sizes=1),
        # a batch of ordinary prompts
        dict(name="prefill_batch", op="prefill", seqs=4, q_heads=32, kv_heads=8, dim=128,
             len_lo=2048, len_hi=2048, sizes=2),
        # one long prompt of odd length
        dict(name="prefill_long", op="prefill", seqs=1, q_heads=32, kv_heads=8, dim=128,
             len_lo=16381, len_hi=16381, sizes=3),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["slots", "write", "tree", "prefill"])
    sizes = rng.randrange(1 << 20)
    if op == "slots":
        seqs = _log_int(rng, 1, 2048)
        prompts = rng.randint(0, seqs)
        return dict(op=op, seqs=seqs, block=rng.choice([8, 16, 32, 64, 128]),
                    ctx=_log_int(rng, 1, 8192), new=rng.randint(1, 8), prompts=prompts,
                    prompt=_log_int(rng, 1, 511) if prompts else 0, spare=rng.randint(0, 300),
                    sizes=sizes)
    if op == "write":
        q_heads, kv_heads, dim = rng.choice([(32, 8, 128), (24, 4, 256), (16, 2, 128),
                                             (16, 2, 256), (8, 8, 64)])
        most = (131072 * 8 * 128) // (kv_heads * dim) // 2
        rows = _log_int(rng, 1, most)
        return dict(op=op, rows=rows, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    block=rng.choice([8, 16, 32, 64, 128]),
                    layout=rng.choice(["head_major", "token_major"]),
                    skip=rng.randint(0, rows // 2), sizes=sizes)
    if op == "tree":
        q_heads, kv_heads, dim = rng.choice([(32, 8, 128), (24, 4, 256), (16, 2, 128),
                                             (16, 2, 256), (8, 8, 64), (12, 4, 64)])
        seqs = _log_int(rng, 1, 48)
        hi = _log_int(rng, 16, 16384)
        nodes_hi = _log_int(rng, 1, 64)
        return dict(op=op, seqs=seqs, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    block=rng.choice([8, 16, 32, 64]), ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                    nodes_lo=rng.randint(1, nodes_hi), nodes_hi=nodes_hi, sizes=sizes)
    q_heads, kv_heads, dim = rng.choice([(32, 8, 128), (24, 4, 256), (16, 2, 128), (16, 2, 256),
                                         (8, 8, 64), (12, 4, 64)])
    hi = _log_int(rng, 1, 4096)
    return dict(op=op, seqs=_log_int(rng, 1, max(1, min(64, 8192 // hi))), q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, len_lo=rng.randint(1, hi), len_hi=hi, sizes=sizes)


def _slot_sizes(case):
    """(cached tokens, new tokens) of every request."""
    r = random.Random(case["sizes"])
    ctx = [r.randint(0, case["ctx"]) for _ in range(case["seqs"])]
    new = [r.randint(0 if case["new"] > 1 else 1, case["new"]) for _ in range(case["seqs"])]
    for s in r.sample(range(case["seqs"]), case["prompts"]):
        ctx[s] = 0
        new[s] = r.randint(1, case["prompt"])
    return ctx, new


def _tree_sizes(case):
    """(cached tokens before the tree, parents of the tree's nodes) of every request.

    A node's parent is an earlier node (the recent ones more often, as a
    drafter widens a tree level by level) or -1: a first token."""
    r = random.Random(case["sizes"])
    ctx, parents = [], []
    for _ in range(case["seqs"]):
        ctx.append(r.randint(case["ctx_lo"], case["ctx_hi"]))
        n = r.randint(case["nodes_lo"], case["nodes_hi"])
        parents.append([-1 if i == 0 or r.random() < 0.05
                        else min(i - 1, int(i * math.sqrt(r.random()))) for i in range(n)])
    return ctx, parents


def _depths(parents):
    depth = []
    for p in parents:
        depth.append(1 if p < 0 else depth[p] + 1)
    return depth


def _prompt_sizes(case):
    r = random.Random(case["sizes"])
    return [_log_int(r, case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]


def work(case):
    if case["op"] == "slots":
        ctx, new = _slot_sizes(case)
        bs = case["block"]
        rows = sum(new) + case["spare"]
        pages = sum((c + n + bs - 1) // bs - (c + bs - 1) // bs for c, n in zip(ctx, new))
        # in: the two counts per request, the page of each row's old tail, the free pages;
        # out: slot and position per row, offset and length per request, the new entries
        return dict(bytes=4 * (2 * len(ctx) + len(ctx) + pages + 2 * rows + 2 * len(ctx) + pages),
                    flops=0)
    if case["op"] == "write":
        n = case["rows"]
        row = 2 * case["kv_heads"] * case["dim"] * 2
        return dict(bytes=2 * (n - case["skip"]) * row + 4 * n, flops=0)
    D, Hq, Hkv = case["dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "tree":
        ctx, parents = _tree_sizes(case)
        rows = sum(len(p) for p in parents)
        seen = sum(len(p) * c + sum(_depths(p)) for c, p in zip(ctx, parents))
        tokens = sum(ctx) + rows
        pages = sum(-(-(c + len(p)) // case["block"]) for c, p in zip(ctx, parents))
        return dict(bytes=tokens * Hkv * D * 4 + rows * Hq * D * 4 + 4 * (rows + pages),
                    flops=4 * D * Hq * seen)
    lens = _prompt_sizes(case)
    rows = sum(lens)
    return dict(bytes=rows * (Hq * D * 4 + Hkv * D * 4),
                flops=4 * D * Hq * sum(n * (n + 1) // 2 for n in lens))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cumulative(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


def _tables(lens, block, max_blocks, g, spare=0):
    """A page table over a shuffled pool: every request's pages, other
    requests' pages in the entries behind them, and the pool's free pages."""
    pages = [-(-n // block) for n in lens]
    cu = _cumulative(pages)
    pool = torch.randperm(max(1, cu[-1] + spare), generator=g, device=DEV).to(torch.int32)
    at = _i32(cu[:-1])[:, None] + torch.arange(max_blocks, dtype=torch.int32, device=DEV)[None, :]
    return pool[(at % pool.numel()).long()].contiguous(), pool[cu[-1]:].contiguous(), pool.numel()


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(op=case["op"])
    if case["op"] == "slots":
        ctx, new = _slot_sizes(case)
        bs = case["block"]
        need = sum((c + n + bs - 1) // bs - (c + bs - 1) // bs for c, n in zip(ctx, new))
        start = 1 + seed % 5           # pages that earlier steps took from the list
        max_blocks = max(-(-(c + n) // bs) for c, n in zip(ctx, new))
        tables, free, pool = _tables(ctx, bs, max(1, max_blocks), g, spare=need + start + 8)
        rows = sum(new) + case["spare"]
        S = len(ctx)
        st.update(block=bs, pool=pool, tables=tables, free=free, ctx=_i32(ctx), new=_i32(new),
                  start=_i32([start]), end=_i32([0]),
                  slots=torch.zeros(rows, dtype=torch.int32, device=DEV),
                  positions=torch.zeros(rows, dtype=torch.int32, device=DEV),
                  cu=torch.zeros(S + 1, dtype=torch.int32, device=DEV),
                  lens=torch.zeros(S, dtype=torch.int32, device=DEV))
        return st
    if case["op"] == "write":
        n, Hq, Hkv, D, bs = (case[k] for k in ("rows", "q_heads", "kv_heads", "dim", "block"))
        pages = -(-n // bs) + 3
        # K and V as the fused projection of the step leaves them: [rows][Hq + 2 Hkv][D]
        qkv = _normal((n, Hq + 2 * Hkv, D), g)
        shape = (pages, Hkv, bs, D) if case["layout"] == "head_major" else (pages, bs, Hkv, D)
        # whole requests: runs of tokens fill whole pages of a shuffled pool
        page = torch.randperm(pages, generator=g, device=DEV)
        row = torch.arange(n, device=DEV)
        slots = (page[row // bs] * bs + row % bs).to(torch.int32)
        if case["skip"]:
            skip = torch.randperm(n, generator=g, device=DEV)[: case["skip"]]
            slots[skip] = -1
        st.update(layout=case["layout"], block=bs, kv_heads=Hkv, dim=D, pages=pages,
                  k_cache=_normal(shape, g), v_cache=_normal(shape, g), slots=slots, qkv=qkv,
                  k_new=qkv[:, Hq:Hq + Hkv], v_new=qkv[:, Hq + Hkv:])
        return st
    Hq, Hkv, D = case["q_heads"], case["kv_heads"], case["dim"]
    st.update(scale=1.0 / math.sqrt(D))
    if case["op"] == "tree":
        ctx, parents = _tree_sizes(case)
        bs = case["block"]
        lens = [c + len(p) for c, p in zip(ctx, parents)]
        max_blocks = -(-max(lens) // bs)
        tables, _, pool = _tables(lens, bs, max_blocks, g)
        cu = _cumulative(len(p) for p in parents)
        st.update(max_q=max(len(p) for p in parents), tables=tables, lens=_i32(lens), cu=_i32(cu),
                  parents=_i32([p for tree in parents for p in tree]),
                  q=_normal((cu[-1], Hq, D), g), k_cache=_normal((pool, Hkv, bs, D), g),
                  v_cache=_normal((pool, Hkv, bs, D), g),
                  out=torch.zeros((cu[-1], Hq, D), dtype=torch.float16, device=DEV))
        return st
    lens = _prompt_sizes(case)
    cu = _cumulative(lens)
    qkv = _normal((cu[-1], Hq + 2 * Hkv, D), g)
    st.update(max_len=max(lens), cu=_i32(cu), q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv],
              v=qkv[:, Hq + Hkv:],
              out=torch.zeros((cu[-1], Hq, D), dtype=torch.float16, device=DEV))
    return st


# ------------------------------------------------------------------ the plain forms
def _plain_slots(st):
    bs, ctx, new, tables = st["block"], st["ctx"].long(), st["new"].long(), st["tables"]
    S, N = ctx.numel(), st["slots"].numel()
    total = torch.cumsum(new, 0)
    cu = torch.cat([total.new_zeros(1), total])
    lens = ctx + new
    owned = (ctx + bs - 1) // bs
    need = (lens + bs - 1) // bs - owned
    taken = torch.cumsum(need, 0)
    base = st["start"].long() + taken - need
    column = torch.arange(tables.shape[1], device=DEV)[None, :]
    fresh = (column >= owned[:, None]) & (column < (owned + need)[:, None])
    which = (base[:, None] + column - owned[:, None]).clamp(0, st["free"].numel() - 1)
    tables.copy_(torch.where(fresh, st["free"][which], tables))
    row = torch.arange(N, device=DEV)
    seq = torch.searchsorted(total, row, right=True).clamp_(max=S - 1)
    position = ctx[seq] + row - cu[seq]
    page = tables[seq, (position // bs).clamp(0, tables.shape[1] - 1)].long()
    inside = row < total[-1]
    slots = torch.where(inside, page * bs + position % bs, -1)
    positions = torch.where(inside, position, -1)
    end = st["start"].long() + taken[-1]
    return [slots.int(), positions.int(), cu.int(), lens.int(), end.int(), tables]


def _plain_write(st):
    keep = st["slots"] >= 0
    slots = st["slots"][keep].long()
    page, row = slots // st["block"], slots % st["block"]
    k, v = st["k_cache"], st["v_cache"]
    if st["layout"] == "head_major":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    k[page, row] = st["k_new"][keep]
    v[page, row] = st["v_new"][keep]
    return [st["k_cache"], st["v_cache"]]


def _attend(q, k, v, visible, scale):
    """softmax(q k^T scale) v over the visible tokens, fp32: q [S, Hq, n, D], k and v
    [S, Hkv, L, D], visible [S, n, L]; a row that sees nothing is zero."""
    S, Hq, n, D = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    group = Hq // Hkv
    x = (q.float().reshape(S, Hkv, group * n, D) @ k.float().transpose(2, 3)).mul_(scale)
    x = x.view(S, Hkv, group, n, L)
    x.masked_fill_(~visible[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-3e38)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True).clamp_(min=1e-37)
    o = x.view(S, Hkv, group * n, L) @ v.float()
    return (o.view(S, Hkv, group, n, D) / total).reshape(S, Hq, n, D)


def _row_places(cu, rows):
    """(sequence, index within it) of every packed row."""
    row = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(cu[1:].long(), row, right=True)
    return seq, row - cu.long()[seq]


def _padded(x, seq, at, S, n):
    p = x.new_zeros((S, n) + tuple(x.shape[1:]))
    p[seq, at] = x
    return p.transpose(1, 2)


def _plain_tree(st):
    q, cu, lens, n = st["q"], st["cu"], st["lens"].long(), st["max_q"]
    S, bs = lens.numel(), st["k_cache"].shape[2]
    seq, at = _row_places(cu, q.shape[0])
    nodes = (cu[1:] - cu[:-1]).long()
    # ancestors: (I - P)^-1 of the parent matrix P counts the paths, 1 or 0 in a forest
    up = torch.zeros((S, n, n + 1), device=DEV)
    parent = st["parents"].long()
    up[seq, at, torch.where(parent < 0, n, parent)] = 1.0
    eye = torch.eye(n, device=DEV).expand(S, n, n)
    family = torch.linalg.solve_triangular(eye - up[:, :, :n], eye, upper=False,
                                           unitriangular=True) > 0.5
    L = st["tables"].shape[1] * bs
    token = torch.arange(L, device=DEV)
    first = (lens - nodes)[:, None]
    node = token[None, :] - first                               # [S, L]
    in_tree = (node >= 0) & (node < nodes[:, None])
    seen = torch.gather(family, 2, node.clamp(0, n - 1)[:, None, :].expand(S, n, L))
    visible = (node < 0)[:, None, :] | (in_tree[:, None, :] & seen)
    pages = st["tables"].long()
    k = st["k_cache"][pages].transpose(1, 2).reshape(S, -1, L, q.shape[2])
    v = st["v_cache"][pages].transpose(1, 2).reshape(S, -1, L, q.shape[2])
    # what lies behind a request's last token is not its own
    v = v.masked_fill((token[None, :] >= lens[:, None])[:, None, :, None], 0.0)
    o = _attend(_padded(q, seq, at, S, n), k, v, visible, st["scale"])
    return o.transpose(1, 2)[seq, at].half()


def _plain_prefill(st):
    q, cu, n = st["q"], st["cu"], st["max_len"]
    S = cu.numel() - 1
    seq, at = _row_places(cu, q.shape[0])
    causal = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()
    visible = causal.expand(S, n, n)
    o = _attend(_padded(q, seq, at, S, n), _padded(st["k"], seq, at, S, n),
                _padded(st["v"], seq, at, S, n), visible, st["scale"])
    return o.transpose(1, 2)[seq, at].half()


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["op"]
    if own:
        import paged_gqa_decode_03_gb300 as pgd

        if op == "slots":
            pgd.paged_kv_slots(st["slots"], st["cu"], st["lens"], st["end"], st["tables"],
                               st["ctx"], st["new"], st["free"], st["block"], st["pool"],
                               free_start=st["start"], positions=st["positions"])
            return [st["slots"], st["positions"], st["cu"], st["lens"], st["end"], st["tables"]]
        if op == "write":
            layout = None
            if st["layout"] != "head_major":
                layout = (st["kv_heads"], st["block"], st["pages"],
                          pgd.kv_strides(st["layout"], st["kv_heads"], st["block"], st["dim"]))
            pgd.paged_kv_write(st["k_cache"], st["v_cache"], st["k_new"], st["v_new"],
                               st["slots"], layout=layout)
            return [st["k_cache"], st["v_cache"]]
        if op == "tree":
            pgd.paged_gqa_tree(st["out"], st["q"], st["cu"], st["parents"], st["k_cache"],
                               st["v_cache"], st["tables"], st["lens"], st["scale"], st["max_q"])
            return st["out"]
        pgd.packed_gqa_prefill(st["out"], st["q"], st["k"], st["v"], st["cu"], st["scale"],
                               st["max_len"])
        return st["out"]
    if op == "slots":
        return _plain_slots(st)
    if op == "write":
        return _plain_write(st)
    if op == "tree":
        return _plain_tree(st)
    return _plain_prefill(st)


# ------------------------------------------------------------------ in 64 bits
def _exact_rows(q, k, v, scale):
    """One query row per line against its own keys: q [n, G, D], k, v [L, D], all doubles;
    row i of `seen` [n, L] says which."""
    def of(seen):
        z = torch.einsum("ngd,ld->ngl", q, k) * scale
        z = torch.where(seen[:, None, :], z, -math.inf)
        w = torch.exp(z - z.max(dim=2, keepdim=True).values)
        w = torch.where(seen[:, None, :], w, 0.0)
        return torch.einsum("ngl,ld->ngd", w / w.sum(dim=2, keepdim=True), v)
    return of


def exact(case, seed):
    if case["op"] == "slots":
        return None                       # whole numbers
    st = prepare(case, seed)
    if case["op"] == "write":
        D, Hkv, bs = case["dim"], case["kv_heads"], case["block"]
        token_major = case["layout"] == "token_major"
        out = []
        for cache, new in ((st["k_cache"], st["k_new"]), (st["v_cache"], st["v_new"])):
            flat = cache.double().view(-1, D)         # one line per (page, head, row)
            for h in range(Hkv):
                s = st["slots"].long()
                kept = torch.nonzero(s >= 0).view(-1)
                s = s[kept]
                line = s * Hkv + h if token_major else (s // bs * Hkv + h) * bs + s % bs
                flat.index_copy_(0, line, new[kept, h].double())
            out.append(flat.view(cache.shape))
        return out
    if work(case)["flops"] > 6e12:        # doubles run at about 1 TFLOP/s
        return None
    Hq, Hkv, D = case["q_heads"], case["kv_heads"], case["dim"]
    G = Hq // Hkv
    q = st["q"]
    out = torch.zeros((q.shape[0], Hq, D), dtype=torch.float64, device=DEV)
    if case["op"] == "tree":
        ctx, parents = _tree_sizes(case)
        bs, r0 = case["block"], 0
        for s, (c, tree) in enumerate(zip(ctx, parents)):
            n, L = len(tree), c + len(tree)
            pages = st["tables"][s, : -(-L // bs)].long()
            seen = torch.zeros((n, L), dtype=torch.bool)
            seen[:, :c] = True
            for i, p in enumerate(tree):
                if p >= 0:
                    seen[i] = seen[p]
                seen[i, c + i] = True
            seen = seen.to(DEV)
            for g in range(Hkv):
                k = st["k_cache"][pages, g].reshape(-1, D)[:L].double()
                v = st["v_cache"][pages, g].reshape(-1, D)[:L].double()
                rows = q[r0:r0 + n, g * G:(g + 1) * G].double()
                out[r0:r0 + n, g * G:(g + 1) * G] = _exact_rows(rows, k, v, st["scale"])(seen)
            r0 += n
        return out
    r0 = 0
    for n in _prompt_sizes(case):
        for a in range(0, n, 1024):
            b = min(n, a + 1024)
            seen = torch.arange(b, device=DEV)[None, :] <= torch.arange(a, b, device=DEV)[:, None]
            for g in range(Hkv):
                k, v = (st[x][r0:r0 + b, g].double() for x in ("k", "v"))
                rows = q[r0 + a:r0 + b, g * G:(g + 1) * G].double()
                out[r0 + a:r0 + b, g * G:(g + 1) * G] = _exact_rows(rows, k, v, st["scale"])(seen)
        r0 += n
    return out
