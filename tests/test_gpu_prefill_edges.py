"""Packed prompts (packed_gqa_prefill) where their inputs are out of the ordinary: rows of
no prompt in front of the first, weights far below the largest, rows of NaN."""
import math

import numpy as np
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from step_util import assert_attention, attention, packed_seen
from test_gpu_prefill import case, check, run

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("first", [1, 77, 300])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_rows_before_the_first_prompt_stay(D, first, dtype):
    """cu_seqlens that begins above 0: the rows in front hold NaN, are not
    written and reach no prompt; nor are those behind the last."""
    lens = [first, 50, 200, 31]
    c = case(lens, 8, 2, D, seed=51)
    for t in (c["q"], c["k"], c["v"]):
        t[:first] = float("nan")
        t[first + 250:] = float("nan")
    cu = torch.tensor([first, first + 50, first + 250], dtype=torch.int32, device=DEV)
    out = torch.full((sum(lens), 8, D), 7.0, dtype=dtype, device=DEV)
    pgd.packed_gqa_prefill(out, c["q"], c["k"], c["v"], cu, c["scale"], 200)
    torch.cuda.synchronize()
    assert (out[:first] == 7.0).all() and (out[first + 250:] == 7.0).all()
    check(out, c, f"D{D} behind {first} rows", prompts=(1, 2))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_weights_far_below_the_largest(D):
    """The first token takes nearly all of the weight and its V is 0; the others' weights
    are 2^-24.4 of it.  Weights may be off by 2^-11 of themselves or 2^-32 of
    the largest, whichever is more."""
    n = 2000
    c = case([n], 8, 2, D, seed=52)
    q, k, v = (torch.zeros((n, h, D), dtype=torch.float16, device=DEV) for h in (8, 2, 2))
    q[..., 0] = 1.0
    k[1:, :, 0] = -24.375
    v[1:] = 1.0
    c.update(q=q, k=k, v=v, scale=math.log(2))
    out = run(c, dtype=torch.float32)
    ref, A = attention(q, k, v, packed_seen(n), c["scale"])
    lim = (2.0 ** -11 + 2 * (2.0 ** -18 + n * 2.0 ** -24)) * A + n * 2.0 ** -32
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= lim).all(), (err / lim).max()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_nan(D):
    """A query row of NaN gives NaN, no other row notices."""
    c = case([300, 40], 8, 2, D, seed=53)
    c["q"][7, 3] = float("nan")
    c["q"][320] = float("nan")
    out = run(c, dtype=torch.float32)
    assert torch.isnan(out[7, 3]).all() and torch.isnan(out[320]).all()
    keep = torch.ones((340, 8), dtype=torch.bool, device=DEV)
    keep[7, 3] = False
    keep[320] = False
    q = c["q"].masked_fill(~keep[:, :, None], 0.0)
    for rows in (slice(0, 300), slice(300, 340)):
        n = rows.stop - rows.start
        ref, A = attention(q[rows], c["k"][rows], c["v"][rows], packed_seen(n), c["scale"])
        o = torch.where(keep[rows][:, :, None], out[rows], torch.as_tensor(ref, device=DEV).float())
        assert_attention(o, ref, A, n, D, 6.0, f"D{D}")
