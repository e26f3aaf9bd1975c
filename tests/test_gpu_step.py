"""The step's operators in one run, as a serving loop makes them: prompts attended
packed (packed_gqa_prefill), their pages taken and slots made (paged_kv_slots),
their K and V written (paged_kv_write), a tree of drafted tokens appended and
verified (paged_gqa_tree), an accepted path moved to its final places, and the
next decode step over it (paged_gqa_decode) — every result against the dense
64-bit form, also with the first step captured and replayed."""
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from step_util import assert_attention, attention, packed_seen, tree_seen

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Pool:
    """The caches, page tables and free list of a few requests."""

    def __init__(self, S, Hkv, D, BS, pages, max_blocks, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.g, self.S, self.Hkv, self.D, self.BS, self.pages = g, S, Hkv, D, BS, pages
        # what no request owns is NaN: it must never be read
        self.k, self.v = (torch.full((pages, Hkv, BS, D), float("nan"), dtype=torch.float16,
                                     device=DEV) for _ in range(2))
        self.tables = torch.full((S, max_blocks), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        self.start = i32([0])

    def slots(self, context, new, rows):
        o = dict(slots=torch.zeros(rows, dtype=torch.int32, device=DEV),
                 positions=torch.zeros(rows, dtype=torch.int32, device=DEV),
                 cu=torch.zeros(self.S + 1, dtype=torch.int32, device=DEV),
                 lens=torch.zeros(self.S, dtype=torch.int32, device=DEV),
                 end=torch.zeros(1, dtype=torch.int32, device=DEV))
        pgd.paged_kv_slots(o["slots"], o["cu"], o["lens"], o["end"], self.tables, context, new,
                           self.free, self.BS, self.pages, free_start=self.start,
                           positions=o["positions"])
        return o

    def rows(self, n, heads):
        return torch.randn((n, heads, self.D), generator=self.g, device=DEV).half()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("BS", [8, 32])
def test_prompt_tree_accept_decode(D, BS):
    Hq, Hkv, scale = 8, 2, D ** -0.5
    lens = [70, 5, 130]
    trees = [[-1, 0, 0, 1], [-1, -1, 0, 1, 2, 2, 3, 6, 4], [-1]]
    paths = [[0, 1, 3], [0, 2, 5], [0]]
    S, T = 3, sum(lens)
    pool = Pool(S, Hkv, D, BS, 64, 40, seed=D + BS)

    # ---- the prompts: packed attention, pages and slots, writes (a padded launch)
    qkv = pool.rows(T, Hq + 2 * Hkv)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    new, none = i32(lens), i32([0] * S)
    out = torch.zeros((T, Hq, D), dtype=torch.float16, device=DEV)

    def first_step():
        o = pool.slots(none, new, T + 11)
        pgd.packed_gqa_prefill(out, q, k, v, o["cu"], scale, max(lens))
        padded = torch.nn.functional.pad(qkv, (0, 0, 0, 0, 0, 11))
        pgd.paged_kv_write(pool.k, pool.v, padded[:, Hq:Hq + Hkv], padded[:, Hq + Hkv:], o["slots"])
        return o
    o = first_step()
    torch.cuda.synchronize()
    cu = o["cu"].tolist()
    assert cu == [0, 70, 75, 205] and o["lens"].tolist() == lens
    assert (o["slots"][T:] == -1).all()
    for s, n in enumerate(lens):
        r = slice(cu[s], cu[s + 1])
        ref, A = attention(q[r], k[r], v[r], packed_seen(n), scale)
        assert_attention(out[r], ref, A, n, D, float(v[r].abs().max()), f"prompt {s}")
    # the same prompts through the cache
    paged = torch.zeros((T, Hq, D), dtype=torch.float32, device=DEV)
    pgd.paged_gqa_varlen(paged, q.contiguous(), o["cu"], pool.k, pool.v, pool.tables, o["lens"],
                         scale, max(lens))
    torch.cuda.synchronize()
    for s, n in enumerate(lens):
        r = slice(cu[s], cu[s + 1])
        ref, A = attention(q[r], k[r], v[r], packed_seen(n), scale)
        assert_attention(paged[r], ref, A, n, D, float(v[r].abs().max()), f"paged prompt {s}")
    # captured and replayed: the same pages, slots, cache and output
    before = {x: t.clone() for x, t in (("out", out), ("k", pool.k), ("tables", pool.tables))}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = first_step()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, before["out"]) and torch.equal(pool.tables, before["tables"])
    assert torch.equal(pool.k.view(torch.int16), before["k"].view(torch.int16))
    assert torch.equal(again["slots"], o["slots"]) and torch.equal(again["end"], o["end"])

    # ---- drafted trees behind the prompts
    pool.start = o["end"].clone()
    n = [len(t) for t in trees]
    N = sum(n)
    t = pool.slots(o["lens"], i32(n), N)
    tq, tk, tv = pool.rows(N, Hq), pool.rows(N, Hkv), pool.rows(N, Hkv)
    pgd.paged_kv_write(pool.k, pool.v, tk, tv, t["slots"])
    tree_out = torch.zeros((N, Hq, D), dtype=torch.float16, device=DEV)
    pgd.paged_gqa_tree(tree_out, tq, t["cu"], i32(sum(trees, [])), pool.k, pool.v, pool.tables,
                       t["lens"], scale, max(n))
    torch.cuda.synchronize()
    tcu = t["cu"].tolist()
    for s in range(S):
        r, p = slice(tcu[s], tcu[s + 1]), slice(cu[s], cu[s + 1])
        kk, vv = torch.cat([k[p], tk[r]]), torch.cat([v[p], tv[r]])
        ref, A = attention(tq[r], kk, vv, tree_seen(trees[s], lens[s]), scale)
        assert_attention(tree_out[r], ref, A, lens[s] + n[s], D, float(vv.abs().max()), f"tree {s}")

    # ---- the accepted paths move to the first places behind the prompts
    node = [tcu[s] + i for s in range(S) for i in paths[s]]
    place = [tcu[s] + i for s in range(S) for i in range(len(paths[s]))]
    pgd.paged_kv_write(pool.k, pool.v, tk[node], tv[node], t["slots"][place])
    kept = [a + len(p) for a, p in zip(lens, paths)]
    dq = pool.rows(S, Hq)
    dec = torch.zeros((S, Hq, D), dtype=torch.float32, device=DEV)
    pgd.paged_gqa_decode(dec, dq, pool.k, pool.v, pool.tables, i32(kept), scale)
    torch.cuda.synchronize()
    for s in range(S):
        p, a = slice(cu[s], cu[s + 1]), [tcu[s] + i for i in paths[s]]
        kk, vv = torch.cat([k[p], tk[a]]), torch.cat([v[p], tv[a]])
        ref, A = attention(dq[s:s + 1], kk, vv, torch.ones((1, kept[s]), dtype=torch.bool), scale)
        assert_attention(dec[s:s + 1], ref, A, kept[s], D, float(vv.abs().max()), f"decode {s}")
