"""NaN and infinities that one row or token of a latent cache's attention, or of packed latent
prompts, meets: what the formula makes of them there, and every other row and head unchanged.

A key of infinity in its rotated part (which is no value) gives a score of -infinity where the
query's value has the other sign: a weight of 0, the others as without that token; and one of
+infinity where it has the same: infinity - infinity, NaN, in the 64-bit form and here."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from latent_util import LatentCase, assert_attention, attention
from test_gpu_latent_prefill import Prompts

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


def compare(got, ref, A, L, width, vmax, scale, what):
    """NaN exactly where the 64-bit form has it (whole heads of a row), the rest to its bound."""
    nan = np.isnan(ref).all(-1)
    assert (nan == np.isnan(ref).any(-1)).all(), "a row of the form that is NaN in part"
    g = got.detach().cpu().numpy()
    assert (np.isnan(g).all(-1) == nan).all() and (np.isnan(g).any(-1) == nan).all(), what
    ref, A = (np.where(nan[..., None], 0.0, x) for x in (ref, A))
    assert_attention(torch.where(torch.as_tensor(nan, device=got.device)[..., None], 0.0, got), ref, A, L,
                     width, vmax, scale, what)
    return int(nan.sum())


def check_cache(w, out, what):
    count = 0
    for s, L in enumerate(w.lens):
        rows, ref, A = w.expected(s)
        vmax = float(w.rows[s][:, :w.R].abs().max())
        count += compare(out[rows], ref, A, L, w.R + w.P, vmax, w.scale, f"{what} seq {s}")
    return count


# one request of 9000 tokens is cut into pieces over all runs; several short ones share runs
SHAPES = [([9000], [1]), ([9000, 40], [3, 2]), ([600, 600, 130], [2, 2, 5])]


@pytest.mark.parametrize("lens,new", SHAPES)
@pytest.mark.parametrize("R,P,H", [(512, 64, 16), (256, 32, 65), (128, 64, 128)])
def test_a_query_of_nan_stays_in_its_row(lens, new, R, P, H):
    w = LatentCase(lens, new, H, R, P, 16, seed=R + H)
    w.q[0, H // 2, 5] = float("nan")
    w.q_rope[w.T - 1, H - 1, P - 1] = float("nan")
    for dtype in (torch.float32, torch.float16):
        assert check_cache(w, w.run(dtype=dtype), f"{dtype}") == 2


@pytest.mark.parametrize("lens,new", SHAPES)
@pytest.mark.parametrize("R,P,H", [(512, 64, 16), (256, 32, 65)])
@pytest.mark.parametrize("scale", [0.07, -0.07])
def test_scores_of_infinity(lens, new, R, P, H, scale):
    """In the first token, and in one far behind it, of the requests' contexts; heads of either
    sign in every row."""
    w = LatentCase(lens, new, H, R, P, 16, seed=R + H + 1)
    w.scale = scale
    e = P - 3
    for s, at in ((0, 0), (len(lens) - 1, 0), (0, lens[0] * 2 // 3)):
        w.rows[s][at, R + e] = float("inf")
        w.cache[int(w.tables[s, at // 16]), at % 16, R + e] = float("inf")
    # (away from 0, whose product with an infinity is NaN)
    w.q_rope[..., e] = torch.where(w.q_rope[..., e] < 0, w.q_rope[..., e] - 0.25, w.q_rope[..., e] + 0.25)
    count = check_cache(w, w.run(dtype=torch.float32), "infinite")
    assert w.T * H // 8 < count < w.T * H * 7 // 8


def test_scores_that_are_all_of_minus_infinity_give_zeros():
    """Of the one token there is, of every token of a cut request, and of some pieces of one."""
    H, R, P = 16, 512, 64
    w = LatentCase([1, 5000, 5000], [1, 1, 1], H, R, P, 16, seed=21)
    for s, tokens in ((0, range(1)), (1, range(5000)), (2, range(2000, 4500))):
        w.rows[s][list(tokens), R] = float("-inf")
        for j in range(w.tables.shape[1]):
            part = w.rows[s][j * 16:(j + 1) * 16]
            w.cache[int(w.tables[s, j]), :part.shape[0]] = part
    w.q_rope[:, :, 0] = 0.5 + w.q_rope[:, :, 0].abs()
    out = w.run(dtype=torch.float32)
    assert (out[:2] == 0).all()
    rows, ref, A = w.expected(2)
    assert_attention(out[rows], ref, A, 5000, R + P, float(w.rows[2][:, :R].abs().max()), w.scale, "in part")


def test_a_token_of_nan_reaches_its_readers_alone():
    w = LatentCase([3000, 3000, 200], [1, 2, 1], 16, 512, 64, 32, seed=9)
    w.rows[1][1234, 7] = float("nan")
    w.cache[int(w.tables[1, 1234 // 32]), 1234 % 32, 7] = float("nan")
    out = w.run(dtype=torch.float32)
    assert torch.isnan(out[1:3]).all()
    w.check(out, "others", [0, 2])


@pytest.mark.parametrize("D,P,H", [(128, 64, 16), (64, 32, 3)])
def test_prompts_with_queries_of_nan(D, P, H):
    w = Prompts([300, 1, 700], H, D, P, seed=D)
    for row, h, e in ((0, 0, 0), (129, H - 1, D), (299, 0, D + P - 1), (300, 1, 3), (900, H - 1, 2)):
        w.q[row, h, e] = float("nan")
    for dtype in (torch.float32, torch.float16):
        assert check_prompts(w, w.run(dtype=dtype), f"{dtype}") == 5


def check_prompts(w, out, what):
    count, r0 = 0, 0
    for s, n in enumerate(w.lens):
        rows = slice(r0, r0 + n)
        r0 += n
        k = torch.cat([w.k[rows], w.k_rope[rows][:, None].expand(n, w.H, w.P)], -1)
        ref, A = attention(w.q[rows], k, w.v[rows], np.tril(np.ones((n, n), dtype=bool)), w.scale)
        count += compare(out[rows], ref, A, n, w.D + w.P, float(w.v[rows].abs().max()), w.scale,
                         f"{what} prompt {s}")
    return count


@pytest.mark.parametrize("D,P,H", [(128, 64, 16), (64, 32, 3)])
@pytest.mark.parametrize("scale", [0.07, -0.07])
def test_prompts_with_scores_of_infinity(D, P, H, scale):
    """Tokens inside a tile, of the rows behind them alone: those in front do not see them."""
    w = Prompts([300, 700], H, D, P, seed=D + 1)
    w.scale = scale
    for at in (150, 300 + 20, 300 + 511):
        w.k_rope[at, 1] = float("inf")
    q = w.q[..., D + 1]
    w.q[..., D + 1] = torch.where(q < 0, q - 0.25, q + 0.25)
    count = check_prompts(w, w.run(dtype=torch.float32), "infinite")
    assert w.T * H // 8 < count < w.T * H * 7 // 8


def test_prompts_with_keys_and_values_of_nan():
    """A value reaches the rows that follow its token, and those of the same 128 keys; a key the
    rows that follow it."""
    w = Prompts([500], 4, 128, 64, seed=11)
    w.k[260, 2, 5] = float("nan")
    out = w.run(dtype=torch.float32)
    assert torch.isnan(out[260:, 2]).all() and torch.isfinite(out[:260]).all()
    assert torch.isfinite(out[260:, [0, 1, 3]]).all()
    w.check(out, "other heads", heads=[0, 1, 3])
    w.v[300, 1, 7] = float("nan")
    out = w.run(dtype=torch.float32)
    assert torch.isnan(out[300:, 1, 7]).all() and torch.isfinite(out[:256, 1]).all()
    keep = [e for e in range(128) if e != 7]
    assert torch.isfinite(out[:, 1, keep]).all()
