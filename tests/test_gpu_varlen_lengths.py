"""Lengths that the page table cannot hold in paged_gqa_varlen: clamped and
flagged (PGD_DEVERR_SEQ_LEN) as in the decode, in each of its kernels."""
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from paged_gqa_decode_03_gb300.workloads import make_varlen

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


# (head_dim, query tokens): the decode kernel's form, one tile, pairs of tiles
@pytest.mark.parametrize("D,n", [(64, 2), (128, 1), (64, 20), (128, 20), (256, 20), (64, 200),
                                 (128, 200), (256, 200)])
@pytest.mark.parametrize("partition", [0, 256])
def test_length_past_the_table(D, n, partition):
    w = make_varlen(S=3, Hq=8, Hkv=2, D=D, BS=16, ctx=[300, 640 - n, 50], n=[n] * 3, seed=61,
                    device=DEV, poison=False)
    most = w.block_tables.shape[1] * 16
    assert most == 640

    def run(lens):
        out = torch.full((w.total_q, 8, D), 7.0, dtype=torch.float32, device=DEV)
        pgd.paged_gqa_varlen(out, w.q, w.cu_seqlens_q, w.k_cache, w.v_cache, w.block_tables, lens,
                             w.scale, n, kv_partition=partition)
        torch.cuda.synchronize()
        return out
    base = run(w.seq_lens)
    assert pgd.pgd_check_device_error() == 0
    lens = w.seq_lens.clone()
    for bad in (most + 1, 2 ** 31 - 1):
        lens[1] = bad
        assert torch.equal(run(lens), base)      # as the longest one that fits
        assert pgd.pgd_check_device_error() == pgd.DEVERR_SEQ_LEN
    lens[1] = -1
    out = run(lens)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_SEQ_LEN | pgd.DEVERR_QUERY_LEN
    assert (out[n:2 * n] == 7.0).all()
    assert torch.equal(out[:n], base[:n]) and torch.equal(out[2 * n:], base[2 * n:])
