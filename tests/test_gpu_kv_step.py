"""Page tables and slots from token counts (paged_kv_slots) and cache writes by
slot (paged_kv_write), equal to their plain forms, every value."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
import step_util

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
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def step(ctx, new, BS, spare=0, start=2, MB=None, seed=0, free_extra=3):
    rng = np.random.RandomState(seed)
    ctx, new = np.asarray(ctx, dtype=np.int64), np.asarray(new, dtype=np.int64)
    owned, after = -(-ctx // BS), -(-(ctx + new) // BS)
    MB = max(1, int(after.max()) if len(ctx) else 1) if MB is None else MB
    pool = rng.permutation(int(owned.sum() + (after - owned).sum()) + start + free_extra)
    tables = rng.randint(0, len(pool), size=(len(ctx), MB))
    at = 0
    for s in range(len(ctx)):
        tables[s, : owned[s]] = pool[at: at + owned[s]]
        at += owned[s]
    return dict(ctx=ctx, new=new, BS=BS, tables=tables, free=pool[at:], start=start,
                rows=int(new.sum()) + spare, NB=len(pool))


def run(c, positions=True, offset=0):
    """offset: the row outputs start that many words past a 16-byte border."""
    S, N = len(c["ctx"]), c["rows"]
    o = dict(slots=torch.full((N + offset,), 77, dtype=torch.int32, device=DEV)[offset:],
             cu=torch.full((S + 1,), 77, dtype=torch.int32, device=DEV),
             lens=torch.full((S,), 77, dtype=torch.int32, device=DEV),
             end=torch.full((1,), 77, dtype=torch.int32, device=DEV),
             tables=i32(c["tables"]).view(S, -1) if S else
             torch.zeros((0, c["tables"].shape[1]), dtype=torch.int32, device=DEV),
             positions=torch.full((N + offset,), 77, dtype=torch.int32, device=DEV)[offset:]
             if positions else None)
    pgd.paged_kv_slots(o["slots"], o["cu"], o["lens"], o["end"], o["tables"], i32(c["ctx"]),
                       i32(c["new"]), i32(c["free"]), c["BS"], c["NB"],
                       free_start=i32([c["start"]]) if c["start"] else None,
                       positions=o["positions"])
    torch.cuda.synchronize()
    return o


def check(c, o):
    slot, position, cu, lens, end, tables = step_util.slots(
        c["ctx"], c["new"], c["tables"], c["free"], c["start"], c["BS"], c["rows"])
    for got, want in ((o["slots"], slot), (o["cu"], cu), (o["lens"], lens), (o["end"], [end]),
                      (o["tables"], tables), (o["positions"], position)):
        if got is not None:
            assert np.array_equal(got.cpu().numpy(), np.asarray(want))


@pytest.mark.parametrize("BS", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("S", [1, 2, 31, 513, 1500])
def test_slots(BS, S):
    rng = np.random.RandomState(S + BS)
    ctx = rng.randint(0, 4 * BS, S)
    new = rng.randint(0, 9, S)
    new[rng.randint(0, S)] = 700
    ctx[rng.randint(0, S)] = 0
    c = step(ctx, new, BS, spare=int(rng.randint(0, 40)), seed=S)
    check(c, run(c))


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("positions", [True, False])
def test_slots_alignment(offset, positions):
    c = step([5, 0, 16, 31], [4, 9, 1, 2], 16, spare=3, start=0 if offset == 1 else 2)
    check(c, run(c, positions=positions, offset=offset))


def test_slots_edges():
    # no request; no row; requests without new tokens; a page exactly full; one row
    for ctx, new in (([], []), ([0, 5], [0, 0]), ([16, 32], [0, 16]), ([15], [1]), ([16], [1]),
                     ([0], [1])):
        for spare in (0, 5):
            c = step(ctx, new, 16, spare=spare, MB=4)
            check(c, run(c))


def test_slots_most_requests():
    S = pgd.SLOTS_MAX_SEQS
    rng = np.random.RandomState(1)
    c = step(rng.randint(0, 50, S), rng.randint(0, 3, S), 16, spare=100)
    check(c, run(c))


def test_slots_repeats_are_equal():
    c = step(np.arange(100) * 7, np.arange(100) % 5, 8)
    a, b = run(c), run(c)
    assert all(torch.equal(a[k], b[k]) for k in a)
    # again on its own tables: the counts were not advanced, nothing moves
    c2 = dict(c, tables=a["tables"].cpu().numpy())
    check(c, run(c2))


def test_slots_flags():
    # the list runs out: -1 from there on, what was needed is counted
    c = step([0, 0, 0], [20, 20, 20], 16, start=0, free_extra=0)
    c["free"] = c["free"][:3]
    o = run(c)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_NO_PAGE
    s = o["slots"].cpu().numpy()
    assert (s[:36] >= 0).all() and (s[36:] == -1).all() and o["end"].item() == 6
    assert o["tables"].cpu().numpy()[1, 1] == -1 and o["tables"].cpu().numpy()[2, 0] == -1
    # rows that do not fit: left out of cu and lens too, and take no page
    c = step([0, 0, 0], [20, 20, 20], 16, start=0)
    c["rows"] = 25
    o = run(c)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_QUERY_LEN
    assert o["cu"].tolist() == [0, 20, 25, 25] and o["lens"].tolist() == [20, 5, 0]
    want = step_util.slots(c["ctx"], [20, 5, 0], c["tables"], c["free"], 0, 16, 25)
    assert np.array_equal(o["slots"].cpu().numpy(), want[0]) and o["end"].item() == 3
    # past the table
    c = step([30], [10], 16, MB=3)
    c["tables"] = c["tables"][:, :2]
    o = run(c)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_SEQ_LEN
    assert (o["slots"].cpu().numpy()[2:] == -1).all() and o["lens"].item() == 32
    # negative counts count as none
    c = step([5, 5], [3, 3], 16)
    c["ctx"], c["new"] = np.array([-5, 5]), np.array([3, -3])
    o = run(c)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_SEQ_LEN | pgd.DEVERR_QUERY_LEN
    assert o["cu"].tolist() == [0, 3, 3] and o["lens"].tolist() == [3, 5]
    # counts whose sum passes 32 bits
    c = step([0] * 4, [1] * 4, 16, MB=4)
    c["new"] = np.array([2 ** 31 - 1] * 4)
    c["rows"] = 40
    o = run(c)
    assert pgd.pgd_check_device_error() & pgd.DEVERR_QUERY_LEN
    assert o["cu"].tolist() == [0, 40, 40, 40, 40] and o["lens"].tolist() == [40, 0, 0, 0]
    # page ids outside the pool
    c = step([20, 0], [1, 1], 16)
    c["tables"][0, 1] = c["NB"]
    c["free"] = np.full_like(c["free"], -7)
    o = run(c)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_PAGE_RANGE
    assert o["slots"].tolist() == [-1, -1] and o["tables"].cpu().numpy()[1, 0] == -1


# ------------------------------------------------------------------ writes
def write_case(N, Hkv, D, BS, token_major, seed=0, skip=0, pages=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    pages = -(-N // BS) + 3 if pages is None else pages
    shape = (pages, BS, Hkv, D) if token_major else (pages, Hkv, BS, D)
    kc, vc = (torch.randn(shape, generator=g, device=DEV).half() for _ in range(2))
    slots = torch.randperm(pages * BS, generator=g, device=DEV)[:N].to(torch.int32)
    if skip:
        slots[torch.randperm(N, generator=g, device=DEV)[:skip]] = -1
    return kc, vc, slots, g


def plain_write(cache, new, slots, BS, token_major):
    out = cache.clone()
    view = out if token_major else out.transpose(1, 2)
    for n, s in enumerate(slots.tolist()):
        if s >= 0:
            view[s // BS, s % BS] = new[n]
    return out


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hkv", [1, 2, 3, 8])
@pytest.mark.parametrize("BS,token_major", [(8, False), (16, True), (128, False)])
def test_write(D, Hkv, BS, token_major):
    for N in (1, 5, 300):
        kc, vc, slots, g = write_case(N, Hkv, D, BS, token_major, seed=N + D, skip=N // 4)
        # slices of a fused projection's output, and plain rows
        qkv = torch.randn((N, 3 * Hkv, D), generator=g, device=DEV).half()
        for k, v in ((qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]),
                     (qkv[:, :Hkv].contiguous(), qkv[:, Hkv:2 * Hkv].contiguous())):
            k2, v2 = kc.clone(), vc.clone()
            layout = None
            if token_major:
                layout = (Hkv, BS, kc.shape[0], pgd.kv_strides("token_major", Hkv, BS, D))
            pgd.paged_kv_write(k2, v2, k, v, slots, layout=layout)
            torch.cuda.synchronize()
            assert torch.equal(k2, plain_write(kc, k, slots, BS, token_major))
            assert torch.equal(v2, plain_write(vc, v, slots, BS, token_major))


def test_write_padded_layout_touches_nothing_else():
    """Padded pages and rows, K and V interleaved in one allocation."""
    N, Hkv, D, BS, NB = 37, 2, 128, 16, 6
    row, page = D + 24, 2 * Hkv * BS * (D + 24) + 40
    base = torch.randn(NB * page, device=DEV).half()
    want = base.clone()
    k, v = base, base[Hkv * BS * row:]
    strides = (page, BS * row, row)
    slots = torch.randperm(NB * BS, device=DEV)[:N].to(torch.int32)
    new = torch.randn((2, N, Hkv, D), device=DEV).half()
    for n, s in enumerate(slots.tolist()):
        for g in range(Hkv):
            at = (s // BS) * page + g * BS * row + (s % BS) * row
            want[at: at + D] = new[0, n, g]
            want[at + Hkv * BS * row: at + Hkv * BS * row + D] = new[1, n, g]
    # (the last page's V rows end inside the allocation)
    pgd.paged_kv_write(k, v, new[0], new[1], slots, layout=(Hkv, BS, NB, strides))
    torch.cuda.synchronize()
    assert torch.equal(base, want)


def test_write_of_special_values_and_flags():
    kc, vc, slots, g = write_case(20, 2, 64, 8, False, seed=3)
    k = torch.full((20, 2, 64), float("nan"), dtype=torch.float16, device=DEV)
    v = torch.full((20, 2, 64), float("-inf"), dtype=torch.float16, device=DEV)
    bad = slots.clone()
    bad[4] = kc.shape[0] * 8 + 1
    k2, v2 = kc.clone(), vc.clone()
    pgd.paged_kv_write(k2, v2, k, v, bad)
    torch.cuda.synchronize()
    assert pgd.pgd_check_device_error() == pgd.DEVERR_PAGE_RANGE
    keep = slots.clone()
    keep[4] = -1
    assert torch.equal(k2.view(torch.int16), plain_write(kc, k, keep, 8, False).view(torch.int16))
    assert torch.equal(v2.view(torch.int16), plain_write(vc, v, keep, 8, False).view(torch.int16))
    pgd.paged_kv_write(k2, v2, k[:0], v[:0], slots[:0])   # no rows: nothing to do
    torch.cuda.synchronize()


def test_write_past_32_bit_offsets():
    """A cache whose last pages start past element 2^31."""
    Hkv, D, BS = 8, 128, 16
    NB = (2 ** 31 + 2 ** 24) // (Hkv * BS * D)
    kc = torch.zeros((NB, Hkv, BS, D), dtype=torch.float16, device=DEV)
    vc = torch.zeros_like(kc)
    new = torch.randn((3, Hkv, D), device=DEV).half()
    slots = i32([NB * BS - 1, 5, (NB - 2) * BS + 3])
    pgd.paged_kv_write(kc, vc, new, -new, slots)
    torch.cuda.synchronize()
    for n, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // BS, :, s % BS], new[n])
        assert torch.equal(vc[s // BS, :, s % BS], -new[n])
    assert int((kc[-3:] != 0).any(-1).sum()) == 2 * Hkv
