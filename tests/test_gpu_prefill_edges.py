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
