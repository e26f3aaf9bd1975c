"""Tree attention (paged_gqa_tree) where its inputs are out of the ordinary: lengths
that do not fit the page table, rows of NaN, scores that grow from stage to
stage, weights far below the largest, divisions over many sequences, bounds
that are loose.  Plain 64-bit forms and bounds of step_util."""
import math
import random

import numpy as np
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from step_util import assert_attention, attention, bound, tree_seen
from test_gpu_tree import case, check, run

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


def gathered(w, s, L):
    """K and V of sequence s in token order, [L, Hkv, D]."""
    ids = w.block_tables[s, : -(-L // w.BS)].long()
    return [c[ids].transpose(1, 2).reshape(-1, w.Hkv, w.D)[:L] for c in (w.k_cache, w.v_cache)]


def set_keys(w, s, keys):
    """Writes keys [L, Hkv, D] as sequence s's K rows."""
    for t0 in range(0, keys.shape[0], w.BS):
        rows = keys[t0: t0 + w.BS]
        w.k_cache[int(w.block_tables[s, t0 // w.BS]), :, : rows.shape[0]] = rows.transpose(0, 1)


# ------------------------------------------------------------------ lengths
@pytest.mark.parametrize("D,n", [(64, 40), (128, 9), (128, 100), (256, 9), (256, 60)])
def test_length_past_the_table_is_flagged_and_skipped(D, n):
    ctx = [300, 45, 500]
    w, trees, parents = case(ctx, [n, 5, n], 16, 4, D, 16, seed=41)
    most = w.block_tables.shape[1] * 16
    lens, cu = w.seq_lens.clone(), w.cu_seqlens_q.tolist()
    for bad in (most + 1, 2 ** 31 - 1, -1, -2 ** 31):
        lens[1] = bad
        out = torch.full((w.total_q, w.Hq, D), 7.0, dtype=torch.float16, device=DEV)
        pgd.paged_gqa_tree(out, w.q, w.cu_seqlens_q, parents, w.k_cache, w.v_cache,
                           w.block_tables, lens, w.scale, w.max_q_len)
        torch.cuda.synchronize()
        bits = pgd.pgd_check_device_error()
        assert bits & pgd.DEVERR_SEQ_LEN and not bits & ~(pgd.DEVERR_SEQ_LEN | pgd.DEVERR_QUERY_LEN)
        assert (out[cu[1]:cu[2]] == 7.0).all()
        check(out, w, trees, ctx, f"beside a length of {bad}", seqs=(0, 2))
    # the largest length that fits is none of these
    assert int(w.seq_lens.max()) <= most
    run(w, parents)
    assert pgd.pgd_check_device_error() == 0


@pytest.mark.parametrize("bad", [-3, 10 ** 6])
def test_bad_length_of_a_sequence_without_nodes_is_flagged(bad):
    ctx, n = [300, 40, 60], [4, 0, 6]
    w, trees, parents = case(ctx, n, 8, 2, 128, 16, seed=42)
    w.seq_lens[1] = bad
    out = run(w, parents)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_SEQ_LEN
    check(out, w, trees, ctx, "beside it")


# ------------------------------------------------------------------ NaN
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hkv,ctx", [(1, 3000), (4, 60)])
def test_a_row_of_nan_is_nan_whole_or_cut(D, Hkv, ctx):
    """A query row of NaN gives NaN, whether its unit is cut into pieces (one
    KV head, long) or not; no other row notices."""
    n = [9, 70]
    w, trees, parents = case([ctx, ctx + 77], n, 4 * Hkv, Hkv, D, 16, seed=43)
    w.q[3, 1] = float("nan")
    w.q[50] = float("nan")
    out = run(w, parents, dtype=torch.float32)
    assert torch.isnan(out[3, 1]).all() and torch.isnan(out[50]).all()
    keep = torch.ones(out.shape[:2], dtype=torch.bool)
    keep[3, 1] = False
    keep[50] = False
    q = w.q.clone()
    q[3, 1] = q[50] = 0.0
    for s, rows in ((0, slice(0, 9)), (1, slice(9, 79))):
        L = [ctx, ctx + 77][s] + n[s]
        k, v = gathered(w, s, L)
        ref, A = attention(q[rows], k, v, tree_seen(trees[s], L - n[s]), w.scale)
        o = torch.where(keep[rows].to(DEV)[:, :, None], out[rows],
                        torch.as_tensor(ref, device=DEV).float())
        assert_attention(o, ref, A, L, D, float(v.abs().max()), f"sequence {s}", w.scale)


# ------------------------------------------------------------------ moving maxima
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nodes", [3, 30, 70])
@pytest.mark.parametrize("S,ctx", [(1, 700), (9, 2800)])
def test_growing_scores_rescale(D, nodes, S, ctx):
    """Keys that grow along the sequence, so that a row's maximum moves by more
    than 8 (log2) in every stage of 128 tokens: alone in its unit, in pairs of
    tiles (more than 32 nodes of 4 heads), and in units cut between the stages."""
    Hq, Hkv = 8, 2
    w, trees, parents = case([ctx] * S, [nodes] * S, Hq, Hkv, D, 16, seed=44)
    L, stages = ctx + nodes, -(-(ctx + nodes) // 128)
    g = torch.Generator(device=DEV)
    g.manual_seed(D + nodes)
    u = torch.sign(torch.randn((Hkv, D), generator=g, device=DEV))
    w.q[:] = (u.repeat_interleave(4, 0)[None] + 0.05 * torch.randn(w.q.shape, generator=g, device=DEV)).half()
    # a token's score is about scale * D * ramp: 10 log2 units more every 128
    step = 10.0 * math.log(2) / (128 * w.scale * D)
    ramp = torch.arange(L, device=DEV, dtype=torch.float32) * step
    for s in range(S):
        set_keys(w, s, (ramp[:, None, None] * u[None]).half())
    out = run(w, parents, dtype=torch.float32)
    for s in range(S):
        rows = slice(s * nodes, (s + 1) * nodes)
        k, v = gathered(w, s, L)
        seen = tree_seen(trees[s], ctx)
        ref, A = attention(w.q[rows], k, v, seen, w.scale)
        z = torch.einsum("nd,ld->nl", w.q[rows][:, 0].double(), k[:, 0].double()) * w.scale
        z = z.masked_fill(~torch.as_tensor(seen, device=DEV), -torch.inf) / math.log(2)
        tops = torch.stack([z[:, 128 * t: 128 * t + 128].amax(1) for t in range(ctx // 128)], 1)
        assert (tops.diff(dim=1) > 8).all()
        # the score's own rounding (step_util) with sum |q k| scale of these rows
        size = float((w.q[rows].abs().double().sum(2).max() * ramp[-1]) * w.scale) * (1 + 4 / D)
        lim = bound(ref, A, L, D, float(v.abs().max()), False, size / D)
        err = np.abs(out[rows].double().cpu().numpy() - ref)
        assert (err <= lim).all(), f"{(err / lim).max()} times the bound, {stages} stages"


# ------------------------------------------------------------------ small weights
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nodes", [2, 60])
def test_weights_far_below_the_largest(D, nodes):
    """One token takes nearly all of the weight and its V is 0; the others' weights are
    2^-24.4 of it.  Weights may be off by 2^-11 of themselves or 2^-32 of the
    largest, whichever is more."""
    ctx = 2000
    w, trees, parents = case([ctx], [nodes], 8, 2, D, 16, seed=45)
    w.q.zero_()
    w.q[..., 0] = 1.0
    w.base.scale = math.log(2)
    keys = torch.zeros((ctx + nodes, 2, D), dtype=torch.float16, device=DEV)
    keys[1:, :, 0] = -24.375
    set_keys(w, 0, keys)
    w.v_cache.fill_(1.0)
    w.v_cache[int(w.block_tables[0, 0]), :, 0] = 0.0
    out = run(w, parents, dtype=torch.float32)
    k, v = gathered(w, 0, ctx + nodes)
    ref, A = attention(w.q, k, v, tree_seen(trees[0], ctx), w.scale)
    L = ctx + nodes
    lim = (2.0 ** -11 + 2 * (2.0 ** -18 + L * 2.0 ** -24)) * A + L * 2.0 ** -32
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= lim).all(), (err / lim).max()


# ------------------------------------------------------------------ the division of the work
@pytest.mark.parametrize("S", [383, 384, 385, 768, 769, 1300])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 4, 1)])
def test_division_over_many_sequences(S, D, Hq, Hkv):
    """The scan over the sequences takes 384 at a time: one, two, three and four
    rounds; empty sequences lie between the others, at the rounds' borders too."""
    rng = random.Random(S)
    ctx = [rng.choice([0, 3, 128, 129, 500]) for _ in range(S)]
    n = [rng.choice([0, 1, 2, 5, 40]) for _ in range(S)]
    n[0], n[-1] = 2, 3
    if S > 385:
        n[383] = n[384] = 0
    w, trees, parents = case(ctx, n, Hq, Hkv, D, 8, seed=S)
    out = run(w, parents)
    assert torch.isfinite(out).all()
    check(out, w, trees, ctx, f"S {S}",
          seqs=sorted({0, 1, 382, 383 % S, 384 % S, 385 % S, 767 % S, 768 % S, S - 2, S - 1}
                      | set(range(5, S, 97))))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_loose_bound_on_the_nodes(D):
    """max_q_len 256 for trees of at most 8: at head_dim 128 and 256 pairs of CTAs whose
    second tile is empty."""
    ctx, n = [3000, 40, 0, 500], [8, 1, 3, 5]
    w, trees, parents = case(ctx, n, 16, 4, D, 16, seed=46)
    check(run(w, parents, max_q=256), w, trees, ctx, "loose")
