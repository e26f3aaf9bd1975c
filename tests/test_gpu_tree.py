"""Tree attention over the paged cache (paged_gqa_tree) against its plain 64-bit
form, row by row, at the sizes and trees where it can go wrong."""
import random

import numpy as np
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from paged_gqa_decode_03_gb300.workloads import make_varlen
from step_util import assert_attention, attention, tree_seen

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


def random_tree(n, rng, chain=False):
    if chain:
        return [i - 1 for i in range(n)]
    return [-1 if i == 0 or rng.random() < 0.1 else rng.randrange(max(0, i - 6), i)
            for i in range(n)]


def case(ctx, n, Hq, Hkv, D, BS, seed=0, chain=False):
    w = make_varlen(S=len(n), Hq=Hq, Hkv=Hkv, D=D, BS=BS, ctx=ctx, n=n, seed=seed, device=DEV)
    rng = random.Random(seed)
    trees = [random_tree(k, rng, chain) for k in n]
    parents = torch.tensor([p for t in trees for p in t], dtype=torch.int32, device=DEV)
    return w, trees, parents


def run(w, parents, dtype=torch.float16, max_q=None, **kw):
    out = torch.full((w.total_q, w.Hq, w.D), float("nan"), dtype=dtype, device=DEV)
    pgd.paged_gqa_tree(out, w.q, w.cu_seqlens_q, parents, kw.pop("k", w.k_cache),
                       kw.pop("v", w.v_cache), w.block_tables, w.seq_lens, w.scale,
                       w.max_q_len if max_q is None else max_q, **kw)
    torch.cuda.synchronize()
    return out


def check(out, w, trees, ctx, what, seqs=None):
    cu = w.cu_seqlens_q.cpu().numpy()
    for s in range(len(trees)) if seqs is None else seqs:
        n, L = len(trees[s]), ctx[s] + len(trees[s])
        if n == 0:
            continue
        ids = w.block_tables[s, : -(-L // w.BS)].long()
        k, v = (c[ids].transpose(1, 2).reshape(-1, w.Hkv, w.D)[:L] for c in (w.k_cache, w.v_cache))
        rows = slice(cu[s], cu[s + 1])
        ref, A = attention(w.q[rows], k, v, tree_seen(trees[s], ctx[s]), w.scale)
        assert_attention(out[rows], ref, A, L, w.D, float(v.abs().max()), f"{what} seq {s}",
                         w.scale)


CTX = [0, 0, 5, 100, 700, 127, 37, 1000]
NODES = [1, 7, 3, 17, 40, 1, 64, 130]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (16, 2), (4, 4), (24, 4), (5, 1)])
@pytest.mark.parametrize("BS", [8, 16, 128])
def test_shapes(D, Hq, Hkv, BS):
    w, trees, parents = case(CTX, NODES, Hq, Hkv, D, BS, seed=D + Hq + BS)
    check(run(w, parents), w, trees, CTX, f"D{D} {Hq}/{Hkv} BS{BS}")
    assert pgd.pgd_check_device_error() == 0


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 255, 256])
def test_tree_sizes_at_the_word_borders(n):
    ctx = [0, 61, 128, 300]
    w, trees, parents = case(ctx, [n] * 4, 8, 2, 64, 16, seed=n)
    check(run(w, parents), w, trees, ctx, f"n {n}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chain_is_the_causal_form(D):
    ctx, n = [0, 130, 500, 31], [200, 1, 64, 33]
    w, trees, parents = case(ctx, n, 8, 2, D, 16, seed=3, chain=True)
    out = run(w, parents, dtype=torch.float32)
    check(out, w, trees, ctx, "chain")
    plain = torch.empty_like(out)
    pgd.paged_gqa_varlen(plain, w.q, w.cu_seqlens_q, w.k_cache, w.v_cache, w.block_tables,
                         w.seq_lens, w.scale, w.max_q_len)
    torch.cuda.synchronize()
    check(plain, w, trees, ctx, "the causal form")


def test_deep_and_wide_trees():
    """A chain of 256, 256 first tokens, a star, a comb."""
    ctx = [90, 90, 90, 90]
    w = make_varlen(S=4, Hq=4, Hkv=2, D=64, BS=16, ctx=ctx, n=[256] * 4, seed=9, device=DEV)
    trees = [list(range(-1, 255)), [-1] * 256, [-1] + [0] * 255,
             [-1] + [i - 1 if i % 2 else max(0, i - 2) for i in range(1, 256)]]
    parents = torch.tensor(sum(trees, []), dtype=torch.int32, device=DEV)
    check(run(w, parents), w, trees, ctx, "deep and wide")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_work_cut_inside_trees(D, dtype, Hkv):
    """Few heads and long contexts: every unit is cut into many pieces, some of
    them inside its tree, where rows may see nothing of a piece."""
    ctx, n = [4000, 1, 777, 2048 - 13], [40, 130, 7, 256]
    w, trees, parents = case(ctx, n, 4 * Hkv, Hkv, D, 16, seed=D + Hkv)
    check(run(w, parents, dtype=dtype), w, trees, ctx, f"cut D{D}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("S", [1, 3, 400])
def test_many_and_few_sequences(D, S):
    """Runs that hold many units, sequences without nodes between them."""
    rng = random.Random(S)
    ctx = [rng.randrange(0, 300) for _ in range(S)]
    n = [rng.choice([0, 1, 2, 5, 33]) for _ in range(S)]
    n[0] = 3
    w, trees, parents = case(ctx, n, 8, 2, D, 8, seed=S)
    check(run(w, parents), w, trees, ctx, f"S {S}", seqs=range(0, S, 1 if S < 9 else 37))


def test_workspace_layouts_and_repeats():
    ctx, n = [900, 40, 2000], [30, 9, 64]
    w, trees, parents = case(ctx, n, 16, 4, 128, 16, seed=4)
    base = run(w, parents)
    check(base, w, trees, ctx, "base")
    need = pgd.pgd_tree_plan(w.S, w.total_q, w.max_q_len, w.Hq, w.Hkv, w.D, w.BS,
                             w.block_tables.shape[1])
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)   # no initial value needed
    assert torch.equal(run(w, parents, workspace=ws), base)
    with pytest.raises(pgd.PGDError):
        run(w, parents, workspace=ws[: need - 1])
    kt, vt = (c.permute(0, 2, 1, 3).contiguous() for c in (w.k_cache, w.v_cache))
    strides = pgd.kv_strides("token_major", w.Hkv, w.BS, w.D)
    got = run(w, parents, k=kt, v=vt, layout=(w.Hkv, w.BS, w.NB, strides))
    assert torch.equal(got, base)
    for _ in range(3):
        assert torch.equal(run(w, parents), base)


@pytest.mark.parametrize("scale", [-0.07, 0.0, 0.3])
def test_any_scale(scale):
    ctx, n = [0, 200, 31], [70, 5, 130]
    w, trees, parents = case(ctx, n, 8, 2, 128, 16, seed=8)
    w.base.scale = scale
    check(run(w, parents), w, trees, ctx, f"scale {scale}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_output_on_a_16_byte_border(D, dtype):
    ctx, n = [900, 40, 5], [30, 9, 64]
    w, trees, parents = case(ctx, n, 8, 2, D, 16, seed=5)
    base = run(w, parents, dtype=dtype)
    size = base.element_size()
    flat = torch.full((base.numel() + 32,), 7.0, dtype=dtype, device=DEV)
    out = flat[16 // size: 16 // size + base.numel()].view(base.shape)
    pgd.paged_gqa_tree(out, w.q, w.cu_seqlens_q, parents, w.k_cache, w.v_cache, w.block_tables,
                       w.seq_lens, w.scale, w.max_q_len)
    torch.cuda.synchronize()
    assert torch.equal(out, base)
    assert (flat[: 16 // size] == 7.0).all() and (flat[16 // size + base.numel():] == 7.0).all()


def test_two_calls_at_once():
    """Two streams, each with its own scratch and outputs, over the same caches."""
    ctx, n = [3000, 40, 2000, 700], [30, 9, 64, 200]
    w, trees, parents = case(ctx, n, 16, 4, 128, 16, seed=15)
    base = run(w, parents)
    outs = [torch.zeros_like(base) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for o, s in zip(outs, streams):
            pgd.paged_gqa_tree(o, w.q, w.cu_seqlens_q, parents, w.k_cache, w.v_cache,
                               w.block_tables, w.seq_lens, w.scale, w.max_q_len, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, base) for o in outs)


def test_padded_rows_and_empty_sequences_stay():
    """More rows than the sequences own, and a sequence without any."""
    ctx, n = [300, 40, 5, 1200], [4, 0, 6, 50]
    w, trees, parents = case(ctx, n, 8, 2, 128, 16, seed=6)
    for _ in range(2):
        out = torch.full((w.total_q + 9, w.Hq, w.D), 7.0, dtype=torch.float16, device=DEV)
        q = torch.cat([w.q, torch.full((9, w.Hq, w.D), float("nan"), dtype=torch.float16,
                                       device=DEV)])
        pp = torch.cat([parents, torch.full((9,), 3, dtype=torch.int32, device=DEV)])
        pgd.paged_gqa_tree(out, q, w.cu_seqlens_q, pp, w.k_cache, w.v_cache, w.block_tables,
                           w.seq_lens, w.scale, w.max_q_len)
        torch.cuda.synchronize()
        check(out[: w.total_q], w, trees, ctx, "padded")
        assert (out[w.total_q:] == 7.0).all()


def test_flags():
    ctx, n = [50, 60], [8, 9]
    w, trees, parents = case(ctx, n, 8, 2, 128, 16, seed=7)
    bad = parents.clone()
    bad[3], bad[8 + 4] = 3, 100          # itself, and a later node: no parent, flagged
    trees[0][3], trees[1][4] = -1, -1
    out = run(w, bad)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_TREE
    check(out, w, trees, ctx, "bad parents")
    # rows that do not lie inside q: skipped and flagged
    cu = w.cu_seqlens_q.clone()
    cu[2] += 1
    out = torch.full((w.total_q, w.Hq, w.D), float("nan"), dtype=torch.float16, device=DEV)
    pgd.paged_gqa_tree(out, w.q, cu, parents, w.k_cache, w.v_cache, w.block_tables, w.seq_lens,
                       w.scale, 64)
    torch.cuda.synchronize()
    assert pgd.pgd_check_device_error() == pgd.DEVERR_QUERY_LEN
    assert torch.isfinite(out[:8]).all() and torch.isnan(out[8:]).all()


def test_captured_and_replayed_on_another_stream():
    ctx, n = [900, 40, 2000], [30, 9, 64]
    w, trees, parents = case(ctx, n, 16, 4, 128, 16, seed=4)
    base = run(w, parents)
    out = torch.zeros_like(base)

    def call():
        pgd.paged_gqa_tree(out, w.q, w.cu_seqlens_q, parents, w.k_cache, w.v_cache,
                           w.block_tables, w.seq_lens, w.scale, w.max_q_len)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    assert torch.equal(out, base)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, base)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_length_before_rows_of_nan(D):
    """Contexts of 0 to 139 tokens; the rows of the last page behind the sequence
    hold NaN."""
    ctx = list(range(140))
    w, trees, parents = case(ctx, [1 + s % 9 for s in ctx], 4, 2, D, 32, seed=31)
    k, v = w.k_cache.clone(), w.v_cache.clone()
    for s, c in enumerate(ctx):
        L = c + len(trees[s])
        if L % 32:
            page = int(w.block_tables[s, L // 32])
            for t in (k, v):
                t[page, :, L % 32:] = float("nan")
    check(run(w, parents, k=k, v=v), w, trees, ctx, f"D{D}")


def test_pages_past_32_bit_offsets():
    """A cache whose used pages start past element 2^31."""
    ctx, n = [300, 17, 64], [20, 33, 5]
    w, trees, parents = case(ctx, n, 32, 8, 128, 16, seed=32)
    used = w.k_cache.shape[0]
    NB = (2 ** 31 + 2 ** 24) // (8 * 16 * 128) + used
    big = [torch.empty((NB, 8, 16, 128), dtype=torch.float16, device=DEV) for _ in range(2)]
    for t, c in zip(big, (w.k_cache, w.v_cache)):
        t[NB - used:] = c
    out = torch.empty((w.total_q, 32, 128), dtype=torch.float16, device=DEV)
    pgd.paged_gqa_tree(out, w.q, w.cu_seqlens_q, parents, *big, w.block_tables + (NB - used),
                       w.seq_lens, w.scale, w.max_q_len)
    torch.cuda.synchronize()
    check(out, w, trees, ctx, "far pages")
