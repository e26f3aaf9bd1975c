"""paged_rope_write and paged_latent_write refuse queries turned into memory that another
array of the call has, or into rows that overlap, before anything reaches a GPU; arrays that
lie between one another pass."""
import ctypes
import random

import numpy as np
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd

INVALID, NO_DEVICE = 1, 4
N, D, BS, NB = 6, 64, 8, 5
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="with a device the call would be launched")


class Rows:
    """[n, heads, width] halves from half number `at` on."""

    def __init__(self, at, heads, token, head, n=N, width=D):
        self.at, self.heads, self.token, self.head, self.n, self.width = at, heads, token, head, n, width

    def halves(self):
        place = (self.at + self.token * np.arange(self.n)[:, None, None]
                 + self.head * np.arange(self.heads)[None, :, None] + np.arange(self.width))
        return place.ravel()

    @property
    def ptr(self):
        return ctypes.c_void_p((1 << 20) + 2 * self.at)


def apart(i, heads, token=None):
    return Rows((i + 1) << 17, heads, token or heads * D, D)


def rope(q, q_out, k=None, v=None, slots=None, positions=None, inv_freq=None, k_cache=None,
         v_cache=None, cache=(2 * BS * D, BS * D, D)):
    k, v = k or apart(1, 2), v or apart(2, 2)
    far = [slots, positions, inv_freq, k_cache, v_cache]
    s, p, f, kc, vc = (ctypes.c_void_p((1 << 20) + 2 * ((i + 3) << 17)) if at is None else
                       ctypes.c_void_p((1 << 20) + 2 * at) for i, at in enumerate(far))
    return pgd.load_library().paged_rope_write(
        kc, vc, q_out.ptr, q.ptr, k.ptr, v.ptr, s, p, f, ctypes.c_float(1.0), 0, q.n, q.heads, k.heads, D,
        D, BS, NB, *cache, q_out.token, q_out.head, q.token, q.head, k.token, k.head, v.token, v.head,
        None)


def refused(got, *words):
    assert got == INVALID
    message = pgd.load_library().pgd_last_error().decode()
    assert all(w in message for w in words), message


def test_queries_that_reach_over_the_keys():
    """q = q_out = qkv[:, :Hq + Hkv] with k_new = qkv[:, Hq : Hq + Hkv]: a key would be turned in
    place while it is read for the cache."""
    both = Rows(0, 6, 8 * D, D)
    refused(rope(both, both, k=Rows(4 * D, 2, 8 * D, D)), "keys")
    refused(rope(both, both, k=Rows(5 * D, 2, 8 * D, D)), "keys")
    refused(rope(both, both, v=Rows(5 * D, 2, 8 * D, D)), "values")
    # heads between one another, one of them shared
    refused(rope(Rows(0, 4, 12 * D, 3 * D), Rows(0, 4, 12 * D, 3 * D), k=Rows(6 * D, 2, 12 * D, 3 * D)), "keys")


def test_queries_into_another_arrays_memory():
    q, out = apart(0, 4), apart(9, 4)
    last = out.at + N * 4 * D
    refused(rope(q, Rows(q.at + 8, 4, 4 * D, D)), "q_out", "q")
    refused(rope(q, Rows(q.at + 5 * D, 4, 4 * D, D)), "q_out", "q")
    for at in (out.at, last - 2):
        refused(rope(q, out, slots=at), "slots")
        refused(rope(q, out, positions=at), "positions")
        refused(rope(q, out, inv_freq=at), "inv_freq")
    for at in (out.at, out.at - 2 * NB * BS * D + 8, last - 8):
        refused(rope(q, out, k_cache=at), "cache")
        refused(rope(q, out, v_cache=at), "cache")
    # token-major pages
    refused(rope(q, out, k_cache=last - 8, cache=(2 * BS * D, D, 2 * D)), "cache")


def test_rows_of_the_output_that_overlap():
    q = apart(0, 4)
    refused(rope(q, Rows(1 << 20, 4, 4 * D - 8, D)), "rows of q_out")
    refused(rope(q, Rows(1 << 20, 4, 4 * D, D - 8)), "rows of q_out")
    refused(rope(q, Rows(1 << 20, 4, 8, 4 * D)), "rows of q_out")
    refused(rope(q, Rows(1 << 20, 4, 2 * D, 3 * D)), "rows of q_out")     # head 2 of a row, head 0 of the third
    refused(rope(Rows(0, 4, 4 * D, 0 + 8), Rows(0, 4, 4 * D, 8)), "rows of q_out")   # in place


def latent(q, q_out, c=None, k=None, cache=None, strides=(BS * 160, 160)):
    R, P = 128, 32
    at = [(i + 2) << 17 for i in range(6)]
    c = c or Rows(at[0], 1, R + P, R, width=R)
    k = k or Rows(at[0] + R, 1, R + P, P, width=P)
    s, p, f, ca = (ctypes.c_void_p((1 << 20) + 2 * x) for x in at[1:4] + [at[4] if cache is None else cache])
    return pgd.load_library().paged_latent_write(
        ca, q_out.ptr, q.ptr, c.ptr, k.ptr, s, p, f, ctypes.c_float(1.0), 0, q.n, q.heads, R, P, BS, NB,
        *strides, q_out.token, q_out.head, q.token, q.head, c.token, k.token, None)


def test_latent_rows_and_cache():
    P, R = 32, 128
    q = Rows(0, 4, 4 * P, P, width=P)
    refused(latent(q, Rows(P, 4, 4 * P, P, width=P)), "q_out", "q")
    out = Rows(1 << 20, 4, 4 * P, P, width=P)
    refused(latent(q, out, k=Rows((1 << 20) + 3 * P, 1, 4 * P, P, width=P)), "keys")
    refused(latent(q, out, c=Rows((1 << 20) - R + 8, 1, R, R, width=R)), "values")
    end = (1 << 20) + N * 4 * P
    for at in ((1 << 20) - (NB * BS * (R + P) - 8), end - 8):
        refused(latent(q, out, cache=at), "cache")


@no_gpu
def test_arrays_between_one_another_pass():
    """Slices of one projection, heads or rows between one another, neighbours: what is missing
    here is a device."""
    row = 8 * D
    for at in range(0, 8 * D, 2 * D):                       # in place, wherever the queries lie
        q = Rows(at, 2, row, D)
        assert rope(q, q, k=Rows((at + 2 * D) % row, 2, row, D), v=Rows((at + 4 * D) % row, 2, row, D)) == NO_DEVICE
    q = Rows(0, 4, 12 * D, 3 * D)                           # [rows, heads, (q, k, v), D]
    assert rope(q, q, k=Rows(D, 4, 12 * D, 3 * D), v=Rows(2 * D, 4, 12 * D, 3 * D)) == NO_DEVICE
    q = Rows(0, 4, D, N * D)                                # [heads, rows, D]
    assert rope(q, q, k=Rows(4 * N * D, 2, D, N * D)) == NO_DEVICE
    assert rope(q, Rows(N * D * 4, 4, 4 * D, D)) == NO_DEVICE
    q, out = apart(0, 4), apart(9, 4)
    assert rope(q, out, slots=out.at - 2 * N, positions=out.at + N * 4 * D) == NO_DEVICE
    assert rope(q, out, k_cache=out.at - 2 * NB * BS * D, v_cache=out.at + N * 4 * D) == NO_DEVICE
    # rows of q_out in the gaps between pages, and of queries that read one row over and over
    gap = Rows((12 << 17) + 2 * BS * D, 1, 2 * BS * D + D, D, n=NB)
    assert rope(Rows(0, 1, D, D, n=NB), gap, k_cache=12 << 17, cache=(2 * BS * D + D, BS * D, D)) == NO_DEVICE
    assert rope(Rows(0, 4, 8, 8), out) == NO_DEVICE
    # one row: its token stride does not matter
    one = Rows(0, 4, 8, D, n=1)
    assert rope(one, one, k=Rows(4 * D, 2, 8, D, n=1), v=Rows(6 * D, 2, 8, D, n=1)) == NO_DEVICE
    P, R = 32, 128
    q = Rows(R, 4, 4 * (R + P), R + P, width=P)             # the rotary parts of [rows, heads, R + P]
    assert latent(q, q) == NO_DEVICE


@no_gpu
def test_the_check_is_exact():
    """Against the sets of halves of drawn rows."""
    rng = random.Random(7)
    seen = {INVALID: 0, NO_DEVICE: 0}
    for _ in range(4000):
        n = rng.randint(1, 5)

        def rows(heads):
            unit = 8
            return Rows(unit * rng.randint(0, 400), heads, unit * rng.randint(1, 90),
                        rng.choice([D, unit * rng.randint(1, 60)]), n=n)
        q, out, k = rows(rng.randint(1, 3)), rows(1), rows(rng.randint(1, 3))
        out.heads = q.heads
        if rng.random() < 0.5:
            out.token = k.token = q.token
        if rng.random() < 0.5:
            out.head = k.head = q.head
        in_place = out.at == q.at
        if in_place:
            out.token, out.head = q.token, q.head
        w, x, y = out.halves(), q.halves(), k.halves()
        bad = (len(set(w)) < len(w) or (not in_place and bool(set(w) & set(x))) or bool(set(w) & set(y)))
        got = rope(q, out, k=k, v=Rows(1 << 19, k.heads, k.heads * D, D, n=n))
        assert got == (INVALID if bad else NO_DEVICE), (vars(q), vars(out), vars(k))
        seen[got] += 1
    assert min(seen.values()) > 500


@pytest.mark.gpu
def test_heads_between_one_another_are_turned_in_place():
    """q, k and v of a head side by side, queries in place: each as from tensors of their own."""
    import __graft_entry__
    __graft_entry__.build()
    dev, rows, H = "cuda:0", 333, 6
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn((rows, H, 3, D), generator=g, device=dev).half()
    q, k, v = x[:, :, 0], x[:, :, 1], x[:, :, 2]
    slots = torch.randperm(rows, generator=g, device=dev).to(torch.int32)
    pos = torch.arange(rows, device=dev, dtype=torch.int32) * 77
    f, _ = pgd.rope_frequencies(D)
    out = []
    for together in (False, True):
        kc, vc = (torch.zeros((-(-rows // BS), H, BS, D), dtype=torch.float16, device=dev) for _ in "kv")
        qs = q if together else q.contiguous()
        pgd.paged_rope_write(kc, vc, qs, qs, k if together else k.contiguous(),
                             v if together else v.contiguous(), slots, pos, f)
        torch.cuda.synchronize()
        out.append((qs.clone(), kc, vc))
        if not together:
            k0, v0 = k.clone(), v.clone()
    for a, b in zip(*out):
        assert torch.equal(a, b)
    assert torch.equal(k, k0) and torch.equal(v, v0)
    both = torch.cat([q, k], 1)
    with pytest.raises(pgd.PGDError, match="keys"):
        pgd.paged_rope_write(kc, vc, both, both, both[:, H:], v, slots, pos, f)
