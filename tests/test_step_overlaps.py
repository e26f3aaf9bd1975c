"""paged_kv_slots refuses arrays that it writes where they share memory with another
of its arrays, before anything reaches a GPU."""
import ctypes
import itertools

import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd

# in the order of the arguments: the first six are written
VALUES = dict(slots=8, positions=8, cu_seqlens_q=5, seq_lens=4, free_end=1, block_tables=4 * 64,
              context_lens=4, query_lens=4, free_pages=16, free_start=1)
NAMES = list(VALUES)


def call(at):
    return pgd.load_library().paged_kv_slots(*[ctypes.c_void_p(at[n]) for n in NAMES], 4, 8, 16, 16,
                                             64, 1024, ctypes.c_void_p(0))


@pytest.mark.parametrize("a,b", [(a, b) for a, b in itertools.combinations(NAMES, 2)
                                 if NAMES.index(a) < 6])
def test_written_arrays_overlap_nothing(a, b):
    apart = {n: (i + 1) << 20 for i, n in enumerate(NAMES)}
    for at in (apart[b], apart[b] + 4 * (VALUES[b] - 1), apart[b] - 4 * (VALUES[a] - 1)):
        assert call(dict(apart, **{a: at})) == 1
        message = pgd.load_library().pgd_last_error().decode()
        assert "overlaps" in message and a in message and b in message


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a device the call would be launched")
def test_neighbours_pass_the_check():
    """Arrays that only touch (slices of one allocation) are in order: what is
    missing here is a device."""
    at, where = {}, 1 << 20
    for n in NAMES:
        at[n] = where
        where += 4 * VALUES[n]
    assert call(at) == 4
