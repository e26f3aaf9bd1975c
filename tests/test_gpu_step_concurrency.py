"""The step's attention calls at the same time: graphs of their own replayed on
two streams, beside eager calls on a third, all with the library's scratch."""
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
import test_gpu_prefill as prefill
import test_gpu_tree as tree

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


def tree_call(ctx, n, Hq, Hkv, D, seed):
    w, trees, parents = tree.case(ctx, n, Hq, Hkv, D, 16, seed=seed)
    base = tree.run(w, parents)
    tree.check(base, w, trees, ctx, "alone")

    def call(out):
        pgd.paged_gqa_tree(out, w.q, w.cu_seqlens_q, parents, w.k_cache, w.v_cache, w.block_tables,
                           w.seq_lens, w.scale, w.max_q_len)
    return base, call


def prefill_call(lens, Hq, Hkv, D, seed):
    c = prefill.case(lens, Hq, Hkv, D, seed=seed)
    base = prefill.run(c)
    prefill.check(base, c, "alone")

    def call(out):
        pgd.packed_gqa_prefill(out, c["q"], c["k"], c["v"], c["cu"], c["scale"], max(lens))
    return base, call


def captured(call, out):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    return g


@pytest.mark.parametrize("D", [64, 128, 256])
def test_graphs_and_eager_calls_at_once(D):
    """Six calls, units cut into pieces and long lists of units among them, three
    at a time: each gives what it gives alone."""
    calls = [tree_call([3000, 40, 2000, 700], [30, 9, 64, 200], 16, 4, D, 15),
             tree_call([900, 5000], [7, 100], 8, 2, D, 16),
             prefill_call([900, 40, 300], 16, 4, D, 4), prefill_call([64] * 60, 8, 2, D, 5),
             tree_call([100] * 50, [5] * 50, 8, 2, D, 17), prefill_call([700], 8, 2, D, 6)]
    outs = [torch.zeros_like(base) for base, _ in calls]
    graphs = [captured(call, out) for (_, call), out in zip(calls[:4], outs)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for turn in range(4):
        for out in outs:
            out.fill_(7.0)
        torch.cuda.synchronize()
        for i in range(2):
            for k in range(2):          # graphs 0, 1 on one stream, 2, 3 on another
                with torch.cuda.stream(streams[k]):
                    graphs[2 * k + i].replay()
            with torch.cuda.stream(streams[2]):
                calls[4 + i][1](outs[4 + i])
        torch.cuda.synchronize()
        for i, ((base, _), out) in enumerate(zip(calls, outs)):
            assert torch.equal(out, base), f"call {i}, turn {turn}"


@pytest.mark.parametrize("D", [64, 128, 256])
def test_two_graphs_of_one_kind_at_once(D):
    for kind in (lambda seed: tree_call([3000, 40, 2000], [30, 9, 64], 16, 4, D, seed),
                 lambda seed: prefill_call([900, 40, 300], 16, 4, D, seed)):
        calls = [kind(21), kind(22)]
        outs = [torch.zeros_like(base) for base, _ in calls]
        graphs = [captured(call, out) for (_, call), out in zip(calls, outs)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(4):
            for out in outs:
                out.fill_(7.0)
            torch.cuda.synchronize()
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(o, b) for o, (b, _) in zip(outs, calls))
