"""A step over a latent cache, and one with rotary positions over K and V pages, as a
serving loop runs them: the operators one after the other, in streams and in graphs, with
the state of one step read by the next; set-up that fails or is captured; drawn sizes."""
import os
import random
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
import step_util
from latent_util import LatentCase, assert_attention, attention, turned
from test_gpu_latent_prefill import Prompts

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV).half()


class Requests:
    """Requests that grow by new tokens a step, their pages taken from a free list."""

    def __init__(self, context, MB, BS, NB):
        self.S, self.MB, self.BS, self.NB = len(context), MB, BS, NB
        self.context = i32([0] * self.S)
        self.tables = i32(np.zeros((self.S, MB)))
        self.free = torch.randperm(NB, generator=gen(1), device=DEV).to(torch.int32)
        self.start = i32([0])

    def step(self, new, rows):
        """A step's slots, positions, cu and lengths; `rows` holds padding behind the new tokens."""
        S = self.S
        out = dict(slots=i32(np.zeros(rows)), positions=i32(np.zeros(rows)), cu=i32(np.zeros(S + 1)),
                   lens=i32(np.zeros(S)))
        end = i32([0])
        pgd.paged_kv_slots(out["slots"], out["cu"], out["lens"], end, self.tables, self.context,
                           i32(new), self.free, self.BS, self.NB, positions=out["positions"],
                           free_start=self.start)
        self.start, self.context = end, out["lens"]
        return out


def causal(n, L):
    return np.arange(L)[None, :] <= (L - n + np.arange(n))[:, None]


def test_steps_with_rotary_positions():
    """paged_kv_slots -> paged_rope_write -> paged_gqa_varlen: prompts, then tokens, with rows
    of padding in each.  The keys that a step reads were turned by the steps before it."""
    Hq, Hkv, D, BS, MB = 8, 2, 128, 16, 20
    steps = [[100, 7, 0, 33], [1, 1, 5, 1], [3, 0, 1, 2], [1, 1, 1, 1]]
    f, m = pgd.rope_frequencies(96, scaling="by_parts", factor=4.0, original_len=4096)
    q = Requests([0] * 4, MB, BS, 64)
    kc, vc = (torch.zeros((64, Hkv, BS, D), dtype=torch.float16, device=DEV) for _ in "kv")
    kept = [([], []) for _ in range(4)]
    g = gen(2)
    for new in steps:
        n = sum(new)
        rows = n + 3
        qkv = normal((rows, Hq + 2 * Hkv, D), g)
        s = q.step(new, rows)
        queries = qkv[:, :Hq]
        q0, k0, v0 = (x.clone() for x in (queries, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]))
        pgd.paged_rope_write(kc, vc, queries, queries, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:],
                             s["slots"], s["positions"], f, magnitude=m)
        assert torch.equal(queries[n:], q0[n:]), "rows of padding"
        packed = queries.contiguous()
        out = torch.full((rows, Hq, D), float("nan"), device=DEV)
        pgd.paged_gqa_varlen(out, packed, s["cu"], kc, vc, q.tables, s["lens"], D ** -0.5, max(new))
        torch.cuda.synchronize()
        assert torch.isnan(out[n:]).all()
        cu, lens = s["cu"].tolist(), s["lens"].tolist()
        # keys as the write leaves them (fp16 of the rotation in 64 bits, or a neighbour: held
        # to the cache's own bits, which test_gpu_rope holds to the rotation)
        turned_k, tol = turned(k0, s["positions"], f, False, m)
        turned_q, tol_q = turned(q0, s["positions"], f, False, m)
        assert ((packed[:n].double() - turned_q[:n]).abs() <= tol_q[:n]).all()
        for r in range(4):
            a, b = cu[r], cu[r + 1]
            if a == b:
                continue
            at = s["slots"][a:b].long()
            line = kc.transpose(1, 2).reshape(-1, Hkv, D)[at]
            assert ((line.double() - turned_k[a:b]).abs() <= tol[a:b]).all()
            assert s["positions"][a:b].tolist() == list(range(lens[r] - (b - a), lens[r]))
            kept[r][0].append(line)
            kept[r][1].append(v0[a:b])
            k, v = torch.cat(kept[r][0]), torch.cat(kept[r][1])
            ref, A = step_util.attention(packed[a:b], k, v, causal(b - a, lens[r]), D ** -0.5)
            # (turned rows of magnitude m: scores m^2 times as large)
            step_util.assert_attention(out[a:b], ref, A, lens[r], D, float(v.abs().max()),
                                       f"request {r}", scale=m * m * D ** -0.5)


@pytest.mark.parametrize("H,R,P,BS", [(16, 512, 64, 16), (20, 256, 32, 8), (128, 128, 64, 128)])
def test_steps_over_a_latent_cache(H, R, P, BS):
    """paged_kv_slots -> paged_latent_write -> paged_latent_attention, the queries' parts in one
    tensor turned in place; padding behind the last request's rows."""
    steps = [[40, 130, 0, 9], [1, 1, 77, 1], [2, 3, 1, 0], [1, 1, 1, 1]]
    f, _ = pgd.rope_frequencies(P, scaling="linear", factor=2.0)
    q = Requests([0] * 4, -(-160 // BS) + 1, BS, 200)
    cache = torch.full((200, BS, R + P), float("nan"), dtype=torch.float16, device=DEV)
    kept = [[] for _ in range(4)]
    g = gen(3)
    scale = (128 + P) ** -0.5
    for new in steps:
        n = sum(new)
        rows = n + 2
        down = normal((rows, R + P), g)
        qs = normal((rows, H, R + P), g)
        q0 = qs.clone()
        s = q.step(new, rows)
        pgd.paged_latent_write(cache, qs[..., R:], qs[..., R:], down[:, :R], down[:, R:], s["slots"],
                               s["positions"], f, interleaved=True)
        out = torch.full((rows, H, R), float("nan"), dtype=torch.float16, device=DEV)
        single = new == [1] * 4
        pgd.paged_latent_attention(out[:4] if single else out, qs[:4, :, :R] if single else qs[..., :R],
                                   qs[:4, :, R:] if single else qs[..., R:], cache, q.tables,
                                   s["lens"], scale, cu_seqlens_q=None if single else s["cu"],
                                   max_q_len=max(new))
        torch.cuda.synchronize()
        assert torch.isnan(out[n:]).all() and torch.equal(qs[n:], q0[n:])
        assert torch.equal(qs[..., :R], q0[..., :R])
        want, tol = turned(q0[..., R:], s["positions"], f, True)
        assert ((qs[:n, :, R:].double() - want[:n]).abs() <= tol[:n]).all()
        cu, lens = s["cu"].tolist(), s["lens"].tolist()
        for r in range(4):
            a, b = cu[r], cu[r + 1]
            if a == b:
                continue
            line = cache.reshape(-1, R + P)[s["slots"][a:b].long()]
            want, tol = turned(down[a:b, None, R:], s["positions"][a:b], f, True)
            assert ((line[:, None, R:].double() - want).abs() <= tol).all()
            assert torch.equal(line[:, :R], down[a:b, :R])
            kept[r].append(line)
            k = torch.cat(kept[r])[:, None]
            ref, A = attention(qs[a:b], k, k[..., :R], causal(b - a, lens[r]), scale)
            assert_attention(out[a:b], ref, A, lens[r], R + P, float(k.abs().max()), scale, f"request {r}")


def test_absorbed_form_of_expanded_prompts():
    """The two forms of one attention: with keys W_k c and values W_v c of every head, the
    expanded form over them and W_v times the absorbed form over the cache, whose queries are
    W_k^T q, are both held to the 64-bit form over the exact products' fp16."""
    H, R, D, P, BS = 8, 128, 64, 32, 16
    lens = [70, 200, 1]
    g = gen(4)
    T = sum(lens)
    down = normal((T, R + P), g)
    # projections by permutation and sign: their products are exact in fp16
    pick = torch.stack([torch.randperm(R, generator=g, device=DEV)[:D] for _ in range(2 * H)])
    sign = (torch.randint(0, 2, (2 * H, D), generator=g, device=DEV) * 2 - 1).half()
    kv = down[:, :R][:, pick] * sign                                  # [T, 2 H, D]
    q = normal((T, H, D + P), g)
    f, _ = pgd.rope_frequencies(P)
    pos = i32(np.concatenate([np.arange(n) for n in lens]))
    pages = [-(-n // BS) for n in lens]
    tables = i32(np.zeros((3, max(pages))))
    ids = torch.randperm(sum(pages), generator=g, device=DEV).to(torch.int32)
    slots = []
    at = 0
    for s, n in enumerate(lens):
        tables[s, :pages[s]] = ids[at:at + pages[s]]
        at += pages[s]
        t = torch.arange(n, device=DEV)
        slots.append(tables[s, t // BS] * BS + t % BS)
    slots = torch.cat(slots).to(torch.int32)
    cache = torch.full((sum(pages), BS, R + P), float("nan"), dtype=torch.float16, device=DEV)
    pgd.paged_latent_write(cache, q[..., D:], q[..., D:], down[:, :R], down[:, R:], slots, pos, f)
    k_rope = cache.reshape(-1, R + P)[slots.long()][:, R:].contiguous()
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    scale = (D + P) ** -0.5
    expanded = torch.zeros((T, H, D), device=DEV)
    pgd.packed_latent_prefill(expanded, q, kv[:, :H], k_rope, kv[:, H:], cu, scale, max(lens))
    absorbed_q = torch.zeros((T, H, R), dtype=torch.float16, device=DEV)
    for h in range(H):
        absorbed_q[:, h, pick[h]] = q[:, h, :D] * sign[h]
    o = torch.zeros((T, H, R), device=DEV)
    pgd.paged_latent_attention(o, absorbed_q, q[..., D:], cache, tables, i32(lens), scale,
                               cu_seqlens_q=cu, max_q_len=max(lens))
    torch.cuda.synchronize()
    absorbed = torch.stack([o[:, h, pick[H + h]] * sign[H + h] for h in range(H)], 1)
    for s, n in enumerate(lens):
        a = int(cu[s])
        k = torch.cat([kv[a:a + n, :H], k_rope[a:a + n, None].expand(n, H, P)], -1)
        v = kv[a:a + n, H:]
        ref, A = attention(q[a:a + n], k, v, causal(n, n), scale)
        for what, got in (("expanded", expanded), ("absorbed", absorbed)):
            assert_attention(got[a:a + n], ref, A, n, R + P, float(v.abs().max()), scale, f"{what} {s}")


def test_a_captured_step_advances():
    """A whole decode step in a graph, replayed: slots, write and attention of the replay's
    own lengths, with its scratch; between the replays the same call eagerly on another cache."""
    H, R, P, BS, S, NB = 16, 512, 64, 16, 5, 60
    f, _ = pgd.rope_frequencies(P)
    g = gen(5)
    ids = torch.randperm(NB, generator=g, device=DEV).to(torch.int32)
    tables = ids[:S * 10].view(S, 10).contiguous()    # (pages past the first lengths are replaced)
    start = [3, 0, 100, 127, 31]
    w = LatentCase([300, 2000], [1, 1], H, R, P, BS, seed=6)
    beside = w.run(dtype=torch.float32, single=True)
    w.check(beside, "beside")

    def state():
        cache = torch.zeros((NB, BS, R + P), dtype=torch.float16, device=DEV)
        for s, n in enumerate(start):
            x = normal((n, R + P), gen(100 + s))
            for t in range(n):
                cache[int(tables[s, t // BS]), t % BS] = x[t]
        return dict(cache=cache, ctx=i32(start), slots=i32([0] * S), pos=i32([0] * S),
                    cu=i32([0] * (S + 1)), lens=i32([0] * S), end=i32([0]), tables=tables.clone(),
                    new=i32([1] * S), free=ids[S * 10:].contiguous(), start=i32([0]), down=normal((S, R + P), gen(7)),
                    q=normal((S, H, R + P), gen(8)), q_rope=torch.zeros((S, H, P), dtype=torch.float16, device=DEV),
                    out=torch.zeros((S, H, R), device=DEV))

    def step(x):
        pgd.paged_kv_slots(x["slots"], x["cu"], x["lens"], x["end"], x["tables"], x["ctx"], x["new"],
                           x["free"], BS, NB, positions=x["pos"], free_start=x["start"])
        pgd.paged_latent_write(x["cache"], x["q_rope"], x["q"][..., R:], x["down"][:, :R],
                               x["down"][:, R:], x["slots"], x["pos"], f)
        pgd.paged_latent_attention(x["out"], x["q"][..., :R], x["q_rope"], x["cache"], x["tables"],
                                   x["lens"], 0.07)
        x["ctx"].copy_(x["lens"])
        x["start"].copy_(x["end"])
        x["down"].mul_(-0.75)

    eager, replayed = state(), state()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(replayed)
    outs = []
    for _ in range(6):
        step(eager)
        outs.append(eager["out"].clone())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(side):
            graph.replay()
        other = torch.empty_like(beside)
        pgd.paged_latent_attention(other, w.q, w.q_rope, w.cache, w.tables, w.seq_lens, w.scale)
        torch.cuda.synchronize()
        assert torch.equal(replayed["out"], outs[i]), i
        assert torch.equal(other, beside)
    assert torch.equal(replayed["cache"], eager["cache"]) and replayed["lens"].tolist() == [n + 6 for n in start]
    # pages begun on the way: by the requests of 0, 127 and 31 tokens
    assert replayed["end"].tolist() == [3] and pgd.pgd_check_device_error() == 0


def test_calls_at_once():
    """Absorbed and expanded calls, graphs and eager ones, three streams at a time: each
    gives what it gives alone."""
    calls = []
    for i, (lens, new, H, R) in enumerate([([3000, 40, 2000, 700], [3, 1, 2, 5], 16, 512),
                                           ([900, 5000], [1, 1], 128, 512), ([100] * 50, [1] * 50, 8, 128),
                                           ([1, 2, 3], [1, 2, 1], 64, 256)]):
        w = LatentCase(lens, new, H, R, 64, 16, seed=20 + i)
        base = w.run()
        w.check(base, "alone")
        calls.append((base, lambda out, w=w: pgd.paged_latent_attention(
            out, w.q, w.q_rope, w.cache, w.tables, w.seq_lens, w.scale, cu_seqlens_q=w.cu,
            max_q_len=max(w.new))))
    for i, (lens, H, D) in enumerate([([900, 40, 300], 8, 128), ([64] * 40, 4, 64)]):
        c = Prompts(lens, H, D, seed=30 + i)
        base = c.run()
        c.check(base, "alone")
        calls.append((base, lambda out, c=c: pgd.packed_latent_prefill(
            out, c.q, c.k, c.k_rope, c.v, c.cu, c.scale, max(c.lens))))
    outs = [torch.zeros_like(base) for base, _ in calls]
    graphs = []
    for (_, call), out in zip(calls, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(out)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for turn in range(8):
        for out in outs:
            out.fill_(7.0)
        torch.cuda.synchronize()
        for j in range(len(calls)):
            i = (j * 5 + turn) % len(calls)
            with torch.cuda.stream(streams[j % 3]):
                if (j + turn) % 2:
                    graphs[i].replay()
                else:
                    calls[i][1](outs[i])
        torch.cuda.synchronize()
        for i, (base, _) in enumerate(calls):
            assert torch.equal(outs[i], base), (turn, i)


@pytest.mark.parametrize("D", [64, 256])
def test_beside_the_calls_over_k_and_v_pages(D):
    """Calls over latent caches and over K and V pages on three streams: each gives what it
    gives alone."""
    import test_gpu_step_concurrency as other
    w = LatentCase([3000, 700, 64], [2, 1, 3], 16, 512, 64, 16, seed=60)
    c = Prompts([300, 700], 8, 128, seed=61)
    calls = [other.tree_call([3000, 40, 700], [30, 9, 64], 16, 4, D, 62),
             (w.run(), lambda out: pgd.paged_latent_attention(
                 out, w.q, w.q_rope, w.cache, w.tables, w.seq_lens, w.scale, cu_seqlens_q=w.cu,
                 max_q_len=3)),
             other.prefill_call([900, 40, 300], 16, 4, D, 63),
             (c.run(), lambda out: pgd.packed_latent_prefill(
                 out, c.q, c.k, c.k_rope, c.v, c.cu, c.scale, 700))]
    w.check(calls[1][0], "alone")
    c.check(calls[3][0], "alone")
    outs = [torch.zeros_like(base) for base, _ in calls]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for turn in range(6):
        for out in outs:
            out.fill_(7.0)
        torch.cuda.synchronize()
        for i in range(8):
            with torch.cuda.stream(streams[(i + turn) % 3]):
                if i < 4:
                    calls[i][1](outs[i])
                else:                       # the same again, on another stream: its own output
                    calls[i - 4][1](torch.empty_like(outs[i - 4]))
        torch.cuda.synchronize()
        for i, (base, _) in enumerate(calls):
            assert torch.equal(outs[i], base), (turn, i)


def test_prompts_longer_than_any_run():
    """A whole prompt through the absorbed form: many tiles of one request, cut anywhere."""
    w = LatentCase([700], [700], 16, 256, 32, 32, seed=40)
    w.check(w.run(), "one prompt")


@pytest.mark.parametrize("seed", range(12))
def test_drawn_sizes(seed):
    rng = random.Random(seed)
    hi = rng.choice([16, 200, 1500, 6000])
    S = rng.choice([1, 2, 7, 33])
    lens = [rng.randint(0, hi) for _ in range(S)]
    new = [min(n, rng.choice([0, 1, 1, 2, 5, 30])) for n in lens]
    if not sum(new):
        lens[0], new[0] = 5, 2
    H, R = rng.choice([1, 3, 16, 24, 63, 64, 72, 128, 130]), rng.choice([128, 256, 512])
    w = LatentCase(lens, new, H, R, rng.choice([32, 64]), rng.choice([8, 16, 32, 64, 128]), seed=seed,
                   q=rng.choice(["packed", "apart"]), pad_token=rng.choice([0, 8]),
                   pad_page=rng.choice([0, 1]))
    dtype = rng.choice([torch.float16, torch.float32])
    first = w.run(dtype=dtype, max_q=max(new) + rng.choice([0, 3]))
    w.check(first, "drawn")
    assert torch.equal(w.run(dtype=dtype, max_q=max(new)), first)


HEAD = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import pytest
import torch
import paged_gqa_decode_03_gb300 as pgd
from latent_util import LatentCase
from test_gpu_latent_prefill import Prompts
R, D = int(sys.argv[1]), int(sys.argv[2])
w = LatentCase([300, 40, 2000], [3, 1, 2], 16, R, 64, 16, seed=4)
c = Prompts([70, 300], 8, D, seed=3)
"""

FAILED = HEAD + """
for call, check in ((w.run, w.check), (c.run, c.check)):
    pgd.pgd_test_fail_next_set_up()
    with pytest.raises(pgd.PGDError, match="withheld") as e:
        call()
    assert e.value.status == 4
    check(call())
    pgd.pgd_test_fail_next_set_up()
    check(call())                      # set up: nothing to fail
    pgd.pgd_test_fail_next_set_up(False)
assert pgd.pgd_check_device_error() == 0
print("as it should")
"""

CAPTURED = HEAD + """
out = torch.zeros((w.T, w.H, R), dtype=torch.float16, device="cuda:0")
out2 = torch.full((c.T, c.H, D), float("nan"), dtype=torch.float16, device="cuda:0")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    pgd.paged_latent_attention(out, w.q, w.q_rope, w.cache, w.tables, w.seq_lens, w.scale,
                               cu_seqlens_q=w.cu, max_q_len=3)
    pgd.packed_latent_prefill(out2, c.q, c.k, c.k_rope, c.v, c.cu, c.scale, 300)
for _ in range(2):
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    w.check(out, "absorbed")
    c.check(out2, "expanded")
assert pgd.pgd_check_device_error() == 0
print("as it should")
"""


@pytest.mark.parametrize("R,D", [(128, 64), (256, 128), (512, 128)])
@pytest.mark.parametrize("code", ["failed", "captured"])
def test_set_up_in_a_process_of_its_own(R, D, code):
    text = (FAILED if code == "failed" else CAPTURED).format(root=ROOT)
    r = subprocess.run([sys.executable, "-c", text, str(R), str(D)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "as it should" in r.stdout, r.stdout + r.stderr[-3000:]


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_outputs_that_start_on_16_bytes(dtype):
    """16 bytes past a 32-byte boundary, where rows go out in stores of 16 bytes; what lies
    in front and behind is left alone."""
    step = 16 // torch.empty(0, dtype=dtype).element_size()

    def room(shape):
        n = int(np.prod(shape))
        flat = torch.full((n + 4 * step,), 3.0, dtype=dtype, device=DEV)
        assert flat.data_ptr() % 32 == 0
        return flat, flat[step:step + n].view(shape)
    for lens, new, R in (([700, 3], [2, 3], 512), ([129, 5000], [1, 1], 128)):
        w = LatentCase(lens, new, 20, R, 64, 16, seed=50)
        flat, out = room((w.T, w.H, R))
        pgd.paged_latent_attention(out, w.q, w.q_rope, w.cache, w.tables, w.seq_lens, w.scale,
                                   cu_seqlens_q=w.cu, max_q_len=max(new))
        torch.cuda.synchronize()
        w.check(out, "absorbed")
        assert (flat[:step] == 3.0).all() and (flat[step + out.numel():] == 3.0).all()
    for D in (64, 128):
        c = Prompts([130, 300, 1], 3, D, seed=51)
        flat, out = room((c.T, c.H, D))
        pgd.packed_latent_prefill(out, c.q, c.k, c.k_rope, c.v, c.cu, c.scale, 300)
        torch.cuda.synchronize()
        c.check(out, "expanded")
        assert (flat[:step] == 3.0).all() and (flat[step + out.numel():] == 3.0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seed", range(6))
def test_drawn_prompts(D, seed):
    rng = random.Random(100 + seed)
    hi = rng.choice([1, 130, 260, 700, 2500])
    lens = [rng.randint(0 if rng.random() < 0.3 else 1, hi) for _ in range(rng.choice([1, 5, 40]))]
    if not sum(lens):
        lens[0] = 1
    H = rng.choice([1, 3, 8, 20])
    c = Prompts(lens, H, D, rng.choice([32, 64]), seed=seed, between=rng.choice([0, 5]),
                behind=rng.choice([0, 3]))
    dtype = rng.choice([torch.float16, torch.float32])
    first = c.run(dtype=dtype)
    c.check(first, "drawn", heads=sorted({0, H - 1}))
    again = c.run(dtype=dtype, max_len=max(lens) + 7)
    assert torch.equal(torch.nan_to_num(again, nan=9.0), torch.nan_to_num(first, nan=9.0))
