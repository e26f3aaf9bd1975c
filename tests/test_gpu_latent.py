"""Attention over a latent cache (paged_latent_attention) against its plain 64-bit form."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from latent_util import LatentCase

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


LENS = [1, 5, 100, 127, 128, 129, 300, 1000, 64]
NEW = [1, 5, 3, 1, 2, 4, 6, 7, 1]


@pytest.mark.parametrize("R", [128, 256, 512])
@pytest.mark.parametrize("P", [32, 64])
@pytest.mark.parametrize("H", [1, 8, 16, 20, 64, 65, 96, 128])
@pytest.mark.parametrize("BS", [8, 128])
def test_shapes(R, P, H, BS):
    w = LatentCase(LENS, NEW, H, R, P, BS, seed=R + P + H + BS, q="packed" if H % 16 else "heads")
    w.check(w.run(), f"R{R} P{P} H{H} BS{BS}")
    assert pgd.pgd_check_device_error() == 0


@pytest.mark.parametrize("BS", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("H", [16, 128])
def test_single_tokens(BS, H):
    """cu_seqlens_q None: a decode step; a sequence of length 0 gets zeros."""
    lens = [0, 1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1023, 0, 2050]
    w = LatentCase(lens, [1] * len(lens), H, BS=BS, seed=BS + H)
    out = w.run(single=True)
    w.check(out, f"single BS{BS}", [s for s, n in enumerate(lens) if n])
    assert (out[0] == 0).all() and (out[13] == 0).all()
    both = w.run(dtype=torch.float32, single=True)
    w.check(both, f"fp32 BS{BS}", [s for s, n in enumerate(lens) if n])


def test_one_row_of_one_token():
    w = LatentCase([1], [1], 1, 128, 32, 8, seed=1)
    out = w.run(dtype=torch.float32, single=True)
    assert torch.equal(out[0, 0], w.rows[0][0, :128].float())


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("H", [3, 16, 128])
def test_long_and_few(dtype, H):
    """One or two long requests: every unit is cut into many pieces."""
    for lens, new in (([9001], [1]), ([4097, 3], [3, 3]), ([20000, 1], [2, 1])):
        w = LatentCase(lens, new, H, seed=H)
        w.check(w.run(dtype=dtype), f"long {lens}")


@pytest.mark.parametrize("S", [3, 77, 400, 1500])
def test_many_requests(S):
    rng = np.random.default_rng(S)
    lens = [int(x) for x in rng.integers(1, 200, S)]
    new = [int(min(n, k)) for n, k in zip(lens, rng.integers(0, 4, S))]
    w = LatentCase(lens, new, 4, 128, 32, 16, seed=S)
    out = w.run()
    w.check(out, f"S{S}", sorted(set(int(x) for x in rng.integers(0, S, 40))))
    assert torch.isfinite(out).all()


def test_whole_prompts_and_idle_requests():
    """All of a sequence's tokens new (a first row that sees itself alone), and none."""
    w = LatentCase([70, 200, 33, 500], [70, 0, 33, 500], 8, 256, 64, 16, seed=4)
    w.check(w.run(), "prompts")


@pytest.mark.parametrize("n", [1, 2, 7, 64, 65, 130])
@pytest.mark.parametrize("H", [1, 5, 48])
def test_row_tiles(n, H):
    w = LatentCase([n + 50, n, n + 128], [n, n, n], H, 128, 32, 32, seed=n + H)
    w.check(w.run(), f"n{n} H{H}")


@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-6, 0.3])
def test_scales(scale):
    w = LatentCase([300, 17], [2, 1], 16, seed=6)
    w.scale = scale
    w.check(w.run(), f"scale {scale}")


def test_small_weights_beside_a_large_one():
    """One token takes nearly all of the weight; thousands of others share the rest."""
    w = LatentCase([4000], [1], 16, 512, 64, 16, seed=7)
    x = w.rows[0]
    x.mul_(0.05)
    x[1234] = 0
    x[1234, :512] = (w.q[0, 0].float() * 0.35).half()
    for j in range(w.tables.shape[1]):
        w.cache[int(w.tables[0, j])] = x[j * 16:(j + 1) * 16]
    w.check(w.run(dtype=torch.float32), "large weight")


def test_maxima_that_move_in_every_stage():
    w = LatentCase([3000, 3000], [1, 2], 16, 256, 64, 32, seed=8)
    for s in range(2):
        x = w.rows[s]
        x.mul_(torch.linspace(0.05, 3.0, 3000, device=DEV)[:, None].half())
        for j in range(-(-3000 // 32)):
            part = x[j * 32:(j + 1) * 32]
            w.cache[int(w.tables[s, j]), :part.shape[0]] = part
    w.q.copy_((w.q.float() * 0.6 + w.rows[0][-1, :256].float() * 0.1).half())
    out = w.run(dtype=torch.float32)
    # scores reach some 400: the bound's N(0, 1) argument does not hold, so against the
    # weights of the exact scores with the score's own rounding: |dz| <= 2^-23 (R + P)
    # sum_d |q_d k_d| scale
    for s in range(2):
        rows, ref, A = w.expected(s)
        q = torch.cat([w.q[rows], w.q_rope[rows]], -1).double().abs()
        width = (q @ w.rows[s].double().abs().T).max().item() * abs(w.scale)
        tol = (2 * 320 * 2.0 ** -23 * width + 2.0 ** -10 + 2.0 ** -17) * A + 1e-4
        assert (np.abs(out[rows].cpu().numpy() - ref) <= tol).all()


def test_strided_cache():
    w = LatentCase([100, 1000, 7], [1, 3, 2], 16, 512, 64, 16, seed=9, pad_token=8, pad_page=2)
    w.check(w.run(), "padded")


def test_infinite_scores_and_rows_of_nan():
    w = LatentCase([600, 600], [2, 2], 16, 256, 64, 16, seed=10)
    w.q[1, 3, 5] = float("nan")
    out = w.run(dtype=torch.float32)
    assert torch.isnan(out[1, 3]).all()
    ok = torch.ones((4, 16), dtype=torch.bool, device=DEV)
    ok[1, 3] = False
    assert torch.isfinite(out[ok]).all()
    w.q[1, 3, 5] = 0.0
    w.check(torch.where(ok[..., None], out, w.run(dtype=torch.float32)), "others", [1])


def test_device_errors_and_rows_left_alone():
    """(A skipped sequence changes where the others' units are cut, so their results are
    held to the bound, not to the bits of another batch.)"""
    w = LatentCase([300, 300, 300, 300], [2, 2, 2, 2], 8, 256, 32, 16, seed=12)
    MB = w.tables.shape[1]

    def all_but(skipped):
        out = w.run()
        bits = pgd.pgd_check_device_error()
        for s in skipped:
            assert torch.isnan(out[2 * s:2 * s + 2]).all()
        w.check(out, f"all but {skipped}", [s for s in range(4) if s not in skipped])
        return bits
    assert all_but([]) == 0
    w.seq_lens = torch.tensor([300, MB * 16 + 1, -1, 300], dtype=torch.int32, device=DEV)
    assert all_but([1, 2]) == pgd.DEVERR_SEQ_LEN
    w.seq_lens = torch.tensor([300, 1, 300, 300], dtype=torch.int32, device=DEV)   # 2 rows of 1 token
    assert all_but([1]) == pgd.DEVERR_QUERY_LEN
    w.seq_lens = torch.tensor([300] * 4, dtype=torch.int32, device=DEV)
    out = w.run(max_q=1)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_QUERY_LEN and torch.isnan(out).all()
    w.tables[1, 3] = w.NB                             # such a page reads as zeros
    w.tables[3, 2] = -7
    w.rows[1][48:64] = 0
    w.rows[3][32:48] = 0
    assert all_but([]) == pgd.DEVERR_PAGE_RANGE


def test_padded_batch_and_loose_bound():
    w = LatentCase([200, 300], [2, 3], 16, 512, 64, 16, seed=13)
    w.q = torch.cat([w.q, torch.full((4, 16, 512), float("nan"), dtype=torch.float16, device=DEV)])
    w.q_rope = torch.cat([w.q_rope, w.q_rope[:4]])
    w.T = 9
    out = w.run(max_q=100)
    w.check(out, "padded batch")
    assert torch.isnan(out[5:]).all()


def test_caller_workspace_and_streams_and_graphs():
    w = LatentCase([2000, 700, 64], [2, 1, 3], 16, 512, 64, 16, seed=14)
    ref = w.run(dtype=torch.float32)
    w.check(ref, "library scratch")
    need = pgd.pgd_latent_plan(3, 6, 3, 16, 512, 64, 16, w.tables.shape[1])
    ws = torch.full((max(256, need),), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(w.run(dtype=torch.float32, workspace=ws), ref)
    assert torch.equal(w.run(dtype=torch.float32, workspace=ws), ref)      # its old contents do not matter
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert torch.equal(w.run(dtype=torch.float32, stream=side), ref)
    graphs, outs = [], []
    for i in range(2):                               # replayed at the same time
        outs.append(torch.empty_like(ref))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            pgd.paged_latent_attention(outs[i], w.q, w.q_rope, w.cache, w.tables, w.seq_lens,
                                       w.scale, cu_seqlens_q=w.cu, max_q_len=3)
    for _ in range(20):
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    if need:
        with pytest.raises(pgd.PGDError, match="PGD_ERR_WORKSPACE"):
            w.run(workspace=ws[:need - 256])


def test_results_repeat():
    w = LatentCase([3000, 1, 500], [1, 1, 1], 128, seed=15)
    first = w.run(single=True)
    for _ in range(5):
        assert torch.equal(w.run(single=True), first)


def test_cache_past_32_bit_offsets():
    R, P, BS, H = 512, 64, 128, 16
    w = LatentCase([700], [1], H, R, P, BS, seed=16)
    pages = (1 << 31) // (BS * (R + P)) + 40
    big = torch.zeros((pages, BS, R + P), dtype=torch.float16, device=DEV)
    ids = [pages - 1, 3, pages - 17, pages - 2, 0, pages - 30]
    for j, b in enumerate(ids):
        part = w.rows[0][j * BS:(j + 1) * BS]
        big[b, :part.shape[0]] = part
    w.cache, w.tables = big, torch.tensor([ids], dtype=torch.int32, device=DEV)
    w.check(w.run(single=True), "far pages")
