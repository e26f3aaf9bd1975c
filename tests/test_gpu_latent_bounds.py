"""What paged_latent_attention accepts and refuses by the amount of work: a long chunk among
many decode rows over wide tables, and rows that overlap."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from latent_util import LatentCase

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
OK, UNSUPPORTED = 0, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


def plan(S, T, max_q, H, MB, BS=16, R=128, P=32):
    return pgd.load_library().pgd_latent_plan(S, T, max_q, H, R, P, BS, MB, None)


def test_work_is_bounded_by_the_rows_of_the_call():
    """Tables for 131072 tokens are 1024 stages.  256 sequences of at most 2048 rows of 128
    heads would be 2^29 tiles' stages if each had 2048; 2303 rows are 2303 tiles."""
    assert plan(256, 2303, 2048, 128, 8192) == OK
    assert plan(256, 256 * 2048, 2048, 128, 8192) == UNSUPPORTED      # they may all have them
    # one tile of up to 8 rows of 16 heads begins in each of 2^19 sequences
    assert plan((1 << 19) - 1, (1 << 19) - 1, 8, 16, 8192) == OK
    assert plan(1 << 19, 1 << 19, 8, 16, 8192) == UNSUPPORTED
    # more heads than a half tile: two of them a row, or three, with one begun in each sequence
    assert plan(1 << 20, (1 << 19) - 1, 1 << 19, 65, 8192) == OK
    assert plan(100, (1 << 20) // 3 - 50, 1 << 19, 129, 8192) == OK
    assert plan(100, (1 << 20) // 3, 1 << 19, 129, 8192) == UNSUPPORTED
    assert plan(1 << 20, 1 << 19, 1 << 19, 65, 8192) == UNSUPPORTED
    # products that pass 64 bits
    top = (1 << 31) - 1
    assert plan(top, top, top, 65536, 1 << 23, 128) == UNSUPPORTED
    assert plan(top, top, 1, 1, 1 << 23, 128) == UNSUPPORTED
    assert plan(1, top, top, 65536, 1 << 23, 128) == UNSUPPORTED


def test_a_long_chunk_among_many_decode_rows():
    rng = np.random.default_rng(1)
    lens = [2100] + [int(n) for n in rng.integers(1, 300, 255)]
    new = [2048] + [1] * 255
    w = LatentCase(lens, new, 65, 128, 32, 16, seed=3)
    tables = torch.full((256, 8192), -1, dtype=torch.int32, device=DEV)
    tables[:, :w.tables.shape[1]] = w.tables
    w.tables = tables
    out = w.run(max_q=2048)
    assert torch.isfinite(out).all()
    w.check(out, "chunk", [0, 1, 2, 100, 254, 255])
    need = pgd.pgd_latent_plan(256, 2303, 2048, 65, 128, 32, 16, 8192)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(w.run(max_q=2048, workspace=ws), out)
    again = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pgd.paged_latent_attention(again, w.q, w.q_rope, w.cache, w.tables, w.seq_lens, w.scale,
                                   cu_seqlens_q=w.cu, max_q_len=2048)
    for _ in range(2):
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, out)


def test_rows_that_overlap_past_the_count_are_not_run():
    """Offsets 0, 1, 0, 1, ...: half of the sequences have a negative number of rows, the other
    half the same row of 65536 heads, 512 tiles of up to 512 stages: above 2^31 in all."""
    S, H, R, P, BS, MB = 16384, 65536, 128, 32, 128, 512
    cu = torch.tensor([s & 1 for s in range(S + 1)], dtype=torch.int32, device=DEV)
    lens = torch.full((S,), MB * BS, dtype=torch.int32, device=DEV)
    assert (S // 2) * 512 * (MB + 1) > 1 << 31
    tables = torch.zeros((S, MB), dtype=torch.int32, device=DEV)
    cache = torch.zeros((1, BS, R + P), dtype=torch.float16, device=DEV)
    q = torch.zeros((1, H, R), dtype=torch.float16, device=DEV)
    q_rope = torch.zeros((1, H, P), dtype=torch.float16, device=DEV)
    out = torch.full((1, H, R), 7.0, dtype=torch.float16, device=DEV)
    pgd.paged_latent_attention(out, q, q_rope, cache, tables, lens, 0.1, cu_seqlens_q=cu, max_q_len=1)
    torch.cuda.synchronize()
    assert pgd.pgd_check_device_error() == pgd.DEVERR_QUERY_LEN
    assert (out == 7.0).all()
