"""Rotary positions at the cache, and attention over one latent vector a token, as
cases to time.

Four operators of a serving step, each with its plain form in torch:

  rope     a step's queries and keys rotated by their positions, the rotated keys
           and the values into their pages (paged_rope_write)
  latent   the latent cache's counterpart: a token's latent vector and its one
           rotated key into their page, the queries' rotary parts rotated
           (paged_latent_write)
  absorbed attention over the pages of a latent cache, queries taken through the
           keys' projection beforehand (paged_latent_attention)
  expanded causal attention of whole packed prompts with keys and values
           expanded from the latent vectors, one rotary key for all heads
           (packed_latent_prefill)

``own`` False: the plain forms (fp32, angles in 64 bits, rounded once at the end).
``own`` True: the library's entry points.  Sizes follow from the case alone
("sizes" seeds the drawn lengths); the values and the placement of pages follow
from the seed of ``prepare``.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the new token of each request of a decode batch: launch latency
        dict(name="rope_step", op="rope", rows=64, q_heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, block=16, layout="head_major", skip=0, far=8192, sizes=1),
        # a step of mixed prompts in short pages of a token-major cache, a quarter of each
        # head rotated, pairs side by side, far positions, padded rows among them
        dict(name="rope_prompt", op="rope", rows=10007, q_heads=24, kv_heads=4, dim=256, rotary=64,
             interleaved=True, block=8, layout="token_major", skip=500, far=1000000, sizes=2),
        # a long admission: 65 k rows of new prompts
        dict(name="rope_bulk", op="rope", rows=65536, q_heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, block=32, layout="head_major", skip=0, far=131072, sizes=3),
        # a decode batch's new tokens in a latent cache
        dict(name="latent_step", op="latent", rows=128, heads=128, latent=512, rotary=64,
             interleaved=True, block=64, skip=0, far=32768, sizes=1),
        # chunks of prompts in a latent cache, padded rows among them
        dict(name="latent_prompt", op="latent", rows=30011, heads=16, latent=512, rotary=64,
             interleaved=False, block=16, skip=411, far=131072, sizes=2),
        # one request decoding on a slice of the heads: latency
        dict(name="absorbed_one", op="absorbed", seqs=1, heads=16, latent=512, rotary=64, block=16,
             ctx_lo=1000, ctx_hi=1000, new=1, sizes=1),
        # a decode batch with all heads on one GPU
        dict(name="absorbed_batch", op="absorbed", seqs=64, heads=128, latent=512, rotary=64,
             block=32, ctx_lo=512, ctx_hi=4096, new=1, sizes=2),
        # verification of up to five drafted tokens a request
        dict(name="absorbed_verify", op="absorbed", seqs=24, heads=32, latent=512, rotary=64,
             block=16, ctx_lo=100, ctx_hi=8192, new=5, sizes=3),
        # long contexts on a slice of the heads
        dict(name="absorbed_long", op="absorbed", seqs=32, heads=16, latent=512, rotary=64,
             block=64, ctx_lo=8192, ctx_hi=32768, new=1, sizes=4),
        # many short prompts of different lengths, from one token on
        dict(name="expanded_short", op="expanded", seqs=37, heads=16, dim=128, rotary=64, len_lo=1,
             len_hi=512, sizes=1),
        # a batch of ordinary prompts
        dict(name="expanded_batch", op="expanded", seqs=4, heads=32, dim=128, rotary=64,
             len_lo=2048, len_hi=2048, sizes=2),
        # one long prompt of odd length
        dict(name="expanded_long", op="expanded", seqs=1, heads=16, dim=128, rotary=64,
             len_lo=16381, len_hi=16381, sizes=3),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "latent", "absorbed", "expanded"])
    sizes = rng.randrange(1 << 20)
    if op == "rope":
        q_heads, kv_heads, dim = rng.choice([(32, 8, 128), (24, 4, 256), (16, 2, 128),
                                             (16, 2, 256), (8, 8, 64), (5, 1, 64)])
        most = 65536 * 40 * 128 // ((q_heads + 2 * kv_heads) * dim) // 2
        rows = _log_int(rng, 1, most)
        return dict(op=op, rows=rows, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    rotary=16 * rng.randint(1, dim // 16), interleaved=rng.random() < 0.5,
                    block=rng.choice([8, 16, 32, 64, 128]),
                    layout=rng.choice(["head_major", "token_major"]),
                    skip=rng.randint(0, rows // 2), far=_log_int(rng, 16, 4000000), sizes=sizes)
    if op == "latent":
        rows = _log_int(rng, 1, 20000)
        return dict(op=op, rows=rows, heads=rng.choice([1, 8, 16, 20, 32, 64, 128]),
                    latent=rng.choice([128, 256, 512]), rotary=rng.choice([32, 64]),
                    interleaved=rng.random() < 0.5, block=rng.choice([8, 16, 32, 64, 128]),
                    skip=rng.randint(0, rows // 2), far=_log_int(rng, 16, 4000000), sizes=sizes)
    if op == "absorbed":
        hi = _log_int(rng, 16, 16384)
        return dict(op=op, seqs=_log_int(rng, 1, 40), heads=rng.choice([1, 8, 16, 20, 32, 64, 96, 128]),
                    latent=rng.choice([128, 256, 512]), rotary=rng.choice([32, 64]),
                    block=rng.choice([8, 16, 32, 64, 128]), ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                    new=rng.choice([1, 1, 1, 2, 3, 4, 6]), sizes=sizes)
    hi = _log_int(rng, 1, 4096)
    return dict(op=op, seqs=_log_int(rng, 1, max(1, min(64, 8192 // hi))),
                heads=rng.choice([1, 3, 8, 16, 20, 32]), dim=rng.choice([64, 128]),
                rotary=rng.choice([32, 64]), len_lo=rng.randint(1, hi), len_hi=hi, sizes=sizes)


def _positions(case):
    """Runs of consecutive positions: prompts, chunks and single tokens from
    anywhere below "far" on."""
    r = random.Random(case["sizes"])
    out = []
    while len(out) < case["rows"]:
        n = min(case["rows"] - len(out), _log_int(r, 1, 4096))
        start = r.randint(0, case["far"])
        out.extend(range(start, start + n))
    return out


def _request_sizes(case):
    """(cached tokens, new ones among them) of every request."""
    r = random.Random(case["sizes"])
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["seqs"])]
    new = [r.randint(1, case["new"]) for _ in range(case["seqs"])]
    return [c + n for c, n in zip(ctx, new)], new


def _prompt_sizes(case):
    r = random.Random(case["sizes"])
    return [_log_int(r, case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]


def work(case):
    if case["op"] == "rope":
        n, keep = case["rows"], case["rows"] - case["skip"]
        D, rot = case["dim"], case["rotary"]
        # queries and keys in and out, values in and out; a rotation is six operations a pair
        rows = 2 * keep * (case["q_heads"] + 2 * case["kv_heads"]) * D * 2
        return dict(bytes=rows + 8 * n + 2 * rot,
                    flops=3 * keep * (case["q_heads"] + case["kv_heads"]) * rot)
    if case["op"] == "latent":
        n, keep = case["rows"], case["rows"] - case["skip"]
        row = case["latent"] + case["rotary"] * (case["heads"] + 1)
        return dict(bytes=2 * keep * row * 2 + 8 * n + 2 * case["rotary"],
                    flops=3 * keep * (case["heads"] + 1) * case["rotary"])
    if case["op"] == "absorbed":
        lens, new = _request_sizes(case)
        R, P, H = case["latent"], case["rotary"], case["heads"]
        pages = sum(-(-n // case["block"]) for n in lens)
        seen = sum(n * (l - n) + n * (n + 1) // 2 for l, n in zip(lens, new))
        return dict(bytes=sum(lens) * (R + P) * 2 + sum(new) * H * (2 * R + P) * 2 + 4 * pages,
                    flops=2 * H * seen * (2 * R + P))
    lens = _prompt_sizes(case)
    D, P, H = case["dim"], case["rotary"], case["heads"]
    return dict(bytes=sum(lens) * 2 * (H * (4 * D + P) + P),
                flops=2 * H * (2 * D + P) * sum(n * (n + 1) // 2 for n in lens))


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


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)


def _frequencies(rotary):
    """Radians a position of each rotated pair, the ordinary table."""
    return torch.tensor([10000.0 ** (-2.0 * i / rotary) for i in range(rotary // 2)],
                        dtype=torch.float32, device=DEV)


def _rows_to_write(case, pages, g):
    """Slots of whole requests in a shuffled pool and positions; some rows are padding."""
    n, bs = case["rows"], case["block"]
    page = torch.randperm(pages, generator=g, device=DEV)
    row = torch.arange(n, device=DEV)
    slots = (page[row // bs] * bs + row % bs).to(torch.int32)
    positions = _i32(_positions(case))
    if case["skip"]:
        skip = torch.randperm(n, generator=g, device=DEV)[: case["skip"]]
        slots[skip] = -1
        positions[skip] = -1
    return slots, positions


def prepare(case, seed):
    g = _gen(seed)
    st = dict(op=case["op"])
    if case["op"] == "rope":
        n, Hq, Hkv, D, bs = (case[k] for k in ("rows", "q_heads", "kv_heads", "dim", "block"))
        pages = -(-n // bs) + 3
        # as the fused projection of the step leaves them: [rows][Hq + 2 Hkv][D]
        qkv = _normal((n, Hq + 2 * Hkv, D), g)
        shape = (pages, Hkv, bs, D) if case["layout"] == "head_major" else (pages, bs, Hkv, D)
        slots, positions = _rows_to_write(case, pages, g)
        st.update(layout=case["layout"], block=bs, kv_heads=Hkv, dim=D, pages=pages,
                  interleaved=case["interleaved"], k_cache=_normal(shape, g),
                  v_cache=_normal(shape, g), slots=slots, positions=positions,
                  inv_freq=_frequencies(case["rotary"]), q=qkv[:, :Hq], k_new=qkv[:, Hq:Hq + Hkv],
                  v_new=qkv[:, Hq + Hkv:],
                  q_out=torch.zeros((n, Hq, D), dtype=torch.float16, device=DEV))
        return st
    if case["op"] == "latent":
        n, H, R, P, bs = (case[k] for k in ("rows", "heads", "latent", "rotary", "block"))
        pages = -(-n // bs) + 3
        # as the down projection leaves them: [rows][latent + rotary]
        down = _normal((n, R + P), g)
        slots, positions = _rows_to_write(case, pages, g)
        st.update(block=bs, interleaved=case["interleaved"], cache=_normal((pages, bs, R + P), g),
                  slots=slots, positions=positions, inv_freq=_frequencies(P), latent=down[:, :R],
                  k_rope=down[:, R:], q_rope=_normal((n, H, P), g),
                  q_out=torch.zeros((n, H, P), dtype=torch.float16, device=DEV))
        return st
    if case["op"] == "absorbed":
        lens, new = _request_sizes(case)
        H, R, P, bs = (case[k] for k in ("heads", "latent", "rotary", "block"))
        pages = [-(-l // bs) for l in lens]
        cu, at = _cumulative(new), _cumulative(pages)
        pool = torch.randperm(at[-1], generator=g, device=DEV).to(torch.int32)
        entry = _i32(at[:-1])[:, None] + torch.arange(max(pages), dtype=torch.int32, device=DEV)
        # entries behind a request's last page: other requests' pages
        tables = pool[(entry % at[-1]).long()].contiguous()
        # the queries' latent parts as the batched product with the keys' projection
        # leaves them: [heads][rows][latent]
        q = _normal((H, cu[-1], R), g).transpose(0, 1)
        st.update(scale=1.0 / math.sqrt(128 + P), max_q=max(new), single=case["new"] == 1,
                  tables=tables, lens=_i32(lens), cu=_i32(cu), q=q,
                  q_rope=_normal((cu[-1], H, P), g), cache=_normal((at[-1], bs, R + P), g),
                  out=torch.zeros((cu[-1], H, R), dtype=torch.float16, device=DEV))
        return st
    lens = _prompt_sizes(case)
    cu = _cumulative(lens)
    H, D, P = case["heads"], case["dim"], case["rotary"]
    kv = _normal((cu[-1], H, 2 * D), g)          # the up projection's output
    down = _normal((cu[-1], 512 + P), g)         # the down projection's
    st.update(scale=1.0 / math.sqrt(D + P), max_len=max(lens), cu=_i32(cu),
              q=_normal((cu[-1], H, D + P), g), k=kv[:, :, :D], v=kv[:, :, D:],
              k_rope=down[:, 512:],
              out=torch.zeros((cu[-1], H, D), dtype=torch.float16, device=DEV))
    return st


# ------------------------------------------------------------------ the plain forms
def _rotated(x, positions, inv_freq, interleaved):
    """The first 2 * len(inv_freq) values of every head rotated: x [rows, heads, D]."""
    angle = positions.double()[:, None] * inv_freq.double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half = inv_freq.numel()
    y = x.float().clone()
    if interleaved:
        a, b = y[..., 0:2 * half:2].clone(), y[..., 1:2 * half:2].clone()
        y[..., 0:2 * half:2] = a * cos - b * sin
        y[..., 1:2 * half:2] = b * cos + a * sin
    else:
        a, b = y[..., :half].clone(), y[..., half:2 * half].clone()
        y[..., :half] = a * cos - b * sin
        y[..., half:2 * half] = b * cos + a * sin
    return y.to(x.dtype)


def _plain_rope(st):
    keep = st["slots"] >= 0
    at = st["positions"][keep]
    slots = st["slots"][keep].long()
    page, row = slots // st["block"], slots % st["block"]
    k, v = st["k_cache"], st["v_cache"]
    if st["layout"] == "head_major":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    k[page, row] = _rotated(st["k_new"][keep], at, st["inv_freq"], st["interleaved"])
    v[page, row] = st["v_new"][keep]
    st["q_out"][keep] = _rotated(st["q"][keep], at, st["inv_freq"], st["interleaved"])
    return [st["q_out"], st["k_cache"], st["v_cache"]]


def _plain_latent(st):
    keep = st["slots"] >= 0
    at = st["positions"][keep]
    slots = st["slots"][keep].long()
    page, row = slots // st["block"], slots % st["block"]
    R = st["latent"].shape[1]
    key = _rotated(st["k_rope"][keep][:, None], at, st["inv_freq"], st["interleaved"])
    st["cache"][page, row, :R] = st["latent"][keep]
    st["cache"][page, row, R:] = key[:, 0]
    st["q_out"][keep] = _rotated(st["q_rope"][keep], at, st["inv_freq"], st["interleaved"])
    return [st["q_out"], st["cache"]]


def _row_places(cu, rows):
    """(sequence, index within it) of every packed row."""
    row = torch.arange(rows, device=DEV)
    seq = torch.searchsorted(cu[1:].long(), row, right=True)
    return seq, row - cu.long()[seq]


def _softmax(x, visible):
    x.masked_fill_(~visible, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-3e38)
    x = x.sub_(top).exp_()
    return x, x.sum(-1, keepdim=True).clamp_(min=1e-37)


def _plain_absorbed(st):
    q, lens, n = st["q"], st["lens"].long(), st["max_q"]
    T, H, R = q.shape
    S, bs = lens.numel(), st["cache"].shape[1]
    seq, at = _row_places(st["cu"], T)
    count = (st["cu"][1:] - st["cu"][:-1]).long()
    L = st["tables"].shape[1] * bs
    token = torch.arange(L, device=DEV)
    k = st["cache"][st["tables"].long()].reshape(S, L, -1).float()
    # what lies behind a request's last token is not its own
    k.masked_fill_((token[None, :] >= lens[:, None])[:, :, None], 0.0)
    rows = torch.zeros((S, n, H, k.shape[2]), device=DEV)
    rows[seq, at] = torch.cat([q, st["q_rope"]], -1).float()
    x = (rows.view(S, n * H, -1) @ k.transpose(1, 2)).mul_(st["scale"]).view(S, n, H, L)
    last = (lens - count)[:, None] + torch.arange(n, device=DEV)       # a row's own place
    p, total = _softmax(x, (token <= last[:, :, None])[:, :, None, :])
    o = (p.view(S, n * H, L) @ k[:, :, :R]).view(S, n, H, R) / total
    return o[seq, at].half()


def _plain_expanded(st):
    q, cu, n = st["q"], st["cu"], st["max_len"]
    S, H, D = cu.numel() - 1, q.shape[1], st["v"].shape[2]
    seq, at = _row_places(cu, q.shape[0])
    causal = torch.ones((n, n), dtype=torch.bool, device=DEV).tril()

    def padded(x):
        p = torch.zeros((S, n) + tuple(x.shape[1:]), device=DEV)
        p[seq, at] = x.float()
        return p.transpose(1, 2)
    out = torch.empty_like(st["out"])
    step = max(1, min(H, (1 << 30) // (S * n * n)))                    # heads at a time
    shared = padded(st["k_rope"][:, None])
    for h in range(0, H, step):
        a = slice(h, min(H, h + step))
        qh = padded(q[:, a])
        x = qh[..., :D] @ padded(st["k"][:, a]).transpose(2, 3)
        x += qh[..., D:] @ shared.transpose(2, 3)
        p, total = _softmax(x.mul_(st["scale"]), causal)
        o = (p @ padded(st["v"][:, a])).div_(total)
        out[:, a] = o.transpose(1, 2)[seq, at].half()
    return out


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["op"]
    if own:
        import paged_gqa_decode_03_gb300 as pgd

        if op == "rope":
            layout = None
            if st["layout"] != "head_major":
                layout = (st["kv_heads"], st["block"], st["pages"],
                          pgd.kv_strides(st["layout"], st["kv_heads"], st["block"], st["dim"]))
            pgd.paged_rope_write(st["k_cache"], st["v_cache"], st["q_out"], st["q"], st["k_new"],
                                 st["v_new"], st["slots"], st["positions"], st["inv_freq"],
                                 interleaved=st["interleaved"], layout=layout)
            return [st["q_out"], st["k_cache"], st["v_cache"]]
        if op == "latent":
            pgd.paged_latent_write(st["cache"], st["q_out"], st["q_rope"], st["latent"],
                                   st["k_rope"], st["slots"], st["positions"], st["inv_freq"],
                                   interleaved=st["interleaved"])
            return [st["q_out"], st["cache"]]
        if op == "absorbed":
            pgd.paged_latent_attention(st["out"], st["q"], st["q_rope"], st["cache"], st["tables"],
                                       st["lens"], st["scale"],
                                       cu_seqlens_q=None if st["single"] else st["cu"],
                                       max_q_len=st["max_q"])
            return st["out"]
        pgd.packed_latent_prefill(st["out"], st["q"], st["k"], st["k_rope"], st["v"], st["cu"],
                                  st["scale"], st["max_len"])
        return st["out"]
    if op == "rope":
        return _plain_rope(st)
    if op == "latent":
        return _plain_latent(st)
    if op == "absorbed":
        return _plain_absorbed(st)
    return _plain_expanded(st)


# ------------------------------------------------------------------ in 64 bits
def _turned(x, places, freq, interleaved):
    """x [rows, heads, D] in doubles, every pair as one complex number times e^(i angle)."""
    m = freq.numel()
    turn = torch.polar(torch.ones((places.numel(), 1, m), dtype=torch.float64, device=DEV),
                       (places.double()[:, None] * freq.double())[:, None])
    y = x.double()
    part = y[..., :2 * m]
    pairs = part.unflatten(-1, (m, 2)) if interleaved else part.unflatten(-1, (2, m)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, y[..., 2 * m:]], -1)


def _exact_writes(case, st):
    kept = torch.nonzero(st["slots"] >= 0).view(-1)
    s, places = st["slots"][kept].long(), st["positions"][kept]
    if case["op"] == "latent":
        key = _turned(st["k_rope"][kept][:, None], places, st["inv_freq"], case["interleaved"])
        q = st["q_out"].double()
        q.index_copy_(0, kept, _turned(st["q_rope"][kept], places, st["inv_freq"],
                                       case["interleaved"]))
        cache = st["cache"].double()
        cache.view(-1, cache.shape[2]).index_copy_(
            0, s, torch.cat([st["latent"][kept].double(), key[:, 0]], 1))
        return [q, cache]
    D, Hkv, bs = case["dim"], case["kv_heads"], case["block"]
    q = st["q_out"].double()
    q.index_copy_(0, kept, _turned(st["q"][kept], places, st["inv_freq"], case["interleaved"]))
    out = [q]
    for cache, rows in ((st["k_cache"], _turned(st["k_new"][kept], places, st["inv_freq"],
                                                case["interleaved"])),
                        (st["v_cache"], st["v_new"][kept].double())):
        flat = cache.double().view(-1, D)         # one line per (page, head, row)
        for h in range(Hkv):
            line = s * Hkv + h if case["layout"] == "token_major" else \
                (s // bs * Hkv + h) * bs + s % bs
            flat.index_copy_(0, line, rows[:, h])
        out.append(flat.view(cache.shape))
    return out


def _weights(z, seen):
    z = torch.where(seen, z, -math.inf)
    w = torch.where(seen, torch.exp(z - z.amax(-1, keepdim=True)), 0.0)
    return w / w.sum(-1, keepdim=True)


def exact(case, seed):
    if work(case)["flops"] > 4e12:        # doubles run at about 1 TFLOP/s
        return None
    st = prepare(case, seed)
    if case["op"] in ("rope", "latent"):
        return _exact_writes(case, st)
    H = case["heads"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    if case["op"] == "absorbed":
        lens, new = _request_sizes(case)
        R, bs, r0 = case["latent"], case["block"], 0
        for s, (L, n) in enumerate(zip(lens, new)):
            pages = st["tables"][s, : -(-L // bs)].long()
            k = st["cache"][pages].flatten(0, 1)[:L].double()
            z = torch.einsum("nhd,ld->nhl", st["q"][r0:r0 + n].double(), k[:, :R])
            z += torch.einsum("nhd,ld->nhl", st["q_rope"][r0:r0 + n].double(), k[:, R:])
            seen = torch.arange(L, device=DEV) < (L - n + 1 + torch.arange(n, device=DEV))[:, None]
            out[r0:r0 + n] = torch.einsum("nhl,ld->nhd", _weights(z * st["scale"], seen[:, None]),
                                          k[:, :R])
            r0 += n
        return out
    D, r0 = case["dim"], 0
    for n in _prompt_sizes(case):
        for a in range(0, n, 1024):
            b = min(n, a + 1024)
            seen = torch.arange(b, device=DEV)[None, :] <= torch.arange(a, b, device=DEV)[:, None]
            shared = st["k_rope"][r0:r0 + b].double()
            for h in range(H):
                q = st["q"][r0 + a:r0 + b, h].double()
                z = q[:, :D] @ st["k"][r0:r0 + b, h].double().T + q[:, D:] @ shared.T
                out[r0 + a:r0 + b, h] = _weights(z * st["scale"], seen) @ \
                    st["v"][r0:r0 + b, h].double()
        r0 += n
    return out
