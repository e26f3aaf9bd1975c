"""Rotary positions with the write (paged_rope_write, paged_latent_write) against the
rotation in 64 bits, and the cache rows written and left alone."""
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from latent_util import assert_turned, turned

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV).half()


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


def slots_of(n, BS, pages, g):
    return torch.randperm(pages * BS, generator=g, device=DEV)[:n].to(torch.int32)


class GqaRows:
    def __init__(self, N, Hq, Hkv, D, BS, layout="head_major", seed=0, far=100000):
        g = gen(seed)
        self.N, self.Hq, self.Hkv, self.D, self.BS, self.layout = N, Hq, Hkv, D, BS, layout
        self.pages = -(-N // BS) + 3
        qkv = normal((N, Hq + 2 * Hkv, D), g)
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        shape = (self.pages, Hkv, BS, D) if layout == "head_major" else (self.pages, BS, Hkv, D)
        self.kc, self.vc = normal(shape, g), normal(shape, g)
        self.slots = slots_of(N, BS, self.pages, g)
        self.pos = torch.randint(0, far, (N,), generator=g, device=DEV, dtype=torch.int32)
        self.q_out = torch.full((N, Hq, D), 7.0, dtype=torch.float16, device=DEV)

    def cache_layout(self):
        if self.layout == "head_major":
            return None
        return (self.Hkv, self.BS, self.pages,
                pgd.kv_strides(self.layout, self.Hkv, self.BS, self.D))

    def lines(self, cache):
        """[page * BS + row, head, D] view of a cache."""
        c = cache.transpose(1, 2) if self.layout == "head_major" else cache
        return c.reshape(-1, self.Hkv, self.D)

    def run(self, f, **kw):
        pgd.paged_rope_write(self.kc, self.vc, self.q_out, self.q, self.k, self.v, self.slots,
                             self.pos, f, layout=self.cache_layout(), **kw)
        torch.cuda.synchronize()

    def check(self, f, interleaved, magnitude=1.0, before=None, q_in=None):
        k0, v0, q0 = before
        live = self.pos >= 0
        put = live & (self.slots >= 0)
        ref, tol = turned(self.q if q_in is None else q_in, self.pos, f, interleaved, magnitude)
        assert_turned(self.q_out[live], ref[live], tol[live], "q")
        assert torch.equal(self.q_out[~live], q0[~live])
        ref, tol = turned(self.k, self.pos, f, interleaved, magnitude)
        at = self.slots[put].long()
        assert_turned(self.lines(self.kc)[at], ref[put], tol[put], "k")
        assert torch.equal(self.lines(self.vc)[at], self.v[put])
        rest = torch.ones(self.pages * self.BS, dtype=torch.bool, device=DEV)
        rest[at] = False
        assert torch.equal(self.lines(self.kc)[rest], self.lines(k0)[rest])
        assert torch.equal(self.lines(self.vc)[rest], self.lines(v0)[rest])

    def before(self):
        return self.kc.clone(), self.vc.clone(), self.q_out.clone()


@pytest.mark.parametrize("Hq,Hkv,D,rot", [(32, 8, 128, 128), (24, 4, 256, 64), (16, 2, 256, 256),
                                          (5, 1, 64, 64), (8, 8, 64, 16), (16, 2, 128, 48),
                                          (1, 1, 128, 112), (7, 7, 256, 144)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("layout,BS", [("head_major", 16), ("token_major", 8), ("token_major", 128)])
def test_rope_write(Hq, Hkv, D, rot, interleaved, layout, BS):
    w = GqaRows(53, Hq, Hkv, D, BS, layout, seed=D + rot + Hq)
    f, _ = pgd.rope_frequencies(rot)
    w.slots[5::7] = -1
    w.pos[3::11] = -1
    b = w.before()
    w.run(f, interleaved=interleaved)
    w.check(f, interleaved, before=b)
    assert pgd.pgd_check_device_error() == 0


@pytest.mark.parametrize("N", [1, 2, 303, 304, 305, 608, 609, 5000, 20011])
def test_row_counts(N):
    w = GqaRows(N, 8, 2, 128, 16, seed=N)
    f, _ = pgd.rope_frequencies(128)
    b = w.before()
    w.run(f)
    w.check(f, False, before=b)


@pytest.mark.parametrize("far", [1 << 20, 1 << 24, (1 << 31) - 1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(far, interleaved):
    """Angles of 10^9 radians: position and frequency are exact, so is the turn."""
    w = GqaRows(97, 4, 2, 128, 16, seed=11, far=1)
    w.pos = i32([far - i for i in range(97)])
    f, _ = pgd.rope_frequencies(128, base=500000.0)
    b = w.before()
    w.run(f, interleaved=interleaved)
    w.check(f, interleaved, before=b)


def test_frequencies_of_any_sign_and_size():
    """Whole turns drop out of any frequency; negative ones turn backwards."""
    w = GqaRows(64, 4, 2, 64, 16, seed=5, far=4096)
    f = torch.tensor([0.0, 1.0, -1.0, 6.2831855, 7.5, -100.25, 1e-30, 3.1415927, 1e-7, 0.5, -1e-3,
                      12.566371, 2.0, 40.0, 0.1, -0.7], dtype=torch.float32, device=DEV)
    b = w.before()
    w.run(f)
    w.check(f, False, before=b)


@pytest.mark.parametrize("rot", [16, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_magnitude(rot, interleaved):
    w = GqaRows(200, 6, 3, 128, 32, seed=rot)
    f, m = pgd.rope_frequencies(rot, scaling="by_parts", factor=8.0, original_len=2048)
    assert m > 1.2
    q0 = w.q.clone()
    w.q_out = w.q                                    # a slice of the fused projection's output
    w.pos[::9] = -1
    b = w.before()
    k0, v0 = w.k.clone(), w.v.clone()
    w.run(f, interleaved=interleaved, magnitude=m)
    assert torch.equal(w.k, k0) and torch.equal(w.v, v0)
    w.check(f, interleaved, m, before=b, q_in=q0)


def test_keys_alone_and_no_rows():
    w = GqaRows(40, 2, 2, 64, 8, seed=1)
    f, _ = pgd.rope_frequencies(32)
    b = w.before()
    pgd.paged_rope_write(w.kc, w.vc, None, None, w.k, w.v, w.slots, w.pos, f)
    torch.cuda.synchronize()
    w.q_out, _ = turned(w.q, w.pos, f, False)
    w.q_out = w.q_out.half()
    w.check(f, False, before=b)
    k1 = w.kc.clone()
    pgd.paged_rope_write(w.kc, w.vc, None, None, w.k[:0], w.v[:0], w.slots[:0], w.pos[:0], f)
    torch.cuda.synchronize()
    assert torch.equal(w.kc, k1)


def test_strides_of_their_own():
    """q [heads][rows][D], k and v of separate padded buffers, q_out padded."""
    g = gen(3)
    w = GqaRows(77, 6, 2, 64, 16, seed=2)
    w.q = normal((6, 77, 64), g).transpose(0, 1)
    w.k = normal((77, 3, 72), g)[:, :2, :64]
    w.v = normal((77, 2, 128), g)[..., 64:]
    w.q_out = torch.full((77, 9, 80), 7.0, dtype=torch.float16, device=DEV)[:, 2:8, 8:72]
    f, _ = pgd.rope_frequencies(48)
    b = w.before()
    w.run(f, interleaved=True)
    w.check(f, True, before=b)


def test_page_out_of_range_is_flagged():
    w = GqaRows(40, 2, 2, 64, 8, seed=4)
    f, _ = pgd.rope_frequencies(64)
    w.slots[7] = w.pages * w.BS + 3
    b = w.before()
    w.run(f)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_PAGE_RANGE
    w.slots[7] = -1                                  # its queries are turned all the same
    w.check(f, False, before=b)


class LatentRows:
    def __init__(self, N, H, R, P, BS, seed=0, far=100000, pad=0):
        g = gen(seed)
        self.pages = -(-N // BS) + 3
        down = normal((N, R + P), g)
        self.R, self.P, self.BS = R, P, BS
        self.c, self.k = down[:, :R], down[:, R:]
        self.cache = normal((self.pages, BS + (1 if pad else 0), R + P + pad), g)[:, :BS, :R + P]
        self.slots = slots_of(N, BS, self.pages, g)
        self.pos = torch.randint(0, far, (N,), generator=g, device=DEV, dtype=torch.int32)
        self.q = normal((N, H, P), g) if H else None
        self.q_out = torch.full((N, H, P), 7.0, dtype=torch.float16, device=DEV) if H else None

    def run_and_check(self, f, interleaved, magnitude=1.0):
        q0 = None if self.q is None else self.q.clone()
        o0 = None if self.q is None else self.q_out.clone()
        c0 = self.cache.clone()
        pgd.paged_latent_write(self.cache, self.q_out, self.q, self.c, self.k, self.slots, self.pos,
                               f, magnitude=magnitude, interleaved=interleaved)
        torch.cuda.synchronize()
        live = self.pos >= 0
        put = live & (self.slots >= 0) & (self.slots < self.pages * self.BS)
        if q0 is not None:
            ref, tol = turned(q0, self.pos, f, interleaved, magnitude)
            assert_turned(self.q_out[live], ref[live], tol[live], "q")
            assert torch.equal(self.q_out[~live], o0[~live])
        lines, old = self.cache.reshape(-1, self.R + self.P), c0.reshape(-1, self.R + self.P)
        at = self.slots[put].long()
        ref, tol = turned(self.k[:, None], self.pos, f, interleaved, magnitude)
        assert_turned(lines[at][:, None, self.R:], ref[put], tol[put], "k")
        assert torch.equal(lines[at][:, :self.R], self.c[put])
        rest = torch.ones(lines.shape[0], dtype=torch.bool, device=DEV)
        rest[at] = False
        assert torch.equal(lines[rest], old[rest])


@pytest.mark.parametrize("R", [128, 256, 512])
@pytest.mark.parametrize("P", [32, 64])
@pytest.mark.parametrize("H", [0, 1, 20, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_latent_write(R, P, H, interleaved):
    w = LatentRows(61, H, R, P, 8 if H % 2 else 64, seed=R + P + H, pad=8 if R == 256 else 0)
    w.slots[4::9] = -1
    w.pos[6::13] = -1
    f, _ = pgd.rope_frequencies(P)
    w.run_and_check(f, interleaved, 0.75)
    assert pgd.pgd_check_device_error() == 0


@pytest.mark.parametrize("N", [1, 700, 9001])
def test_latent_write_rows_in_place(N):
    w = LatentRows(N, 16, 512, 64, 16, seed=N)
    w.q_out = w.q
    f, _ = pgd.rope_frequencies(64, scaling="base", factor=4.0)
    w.run_and_check(f, True)


def test_latent_page_out_of_range_is_flagged():
    w = LatentRows(40, 2, 128, 32, 8, seed=9)
    w.slots[3] = w.pages * w.BS
    w.run_and_check(pgd.rope_frequencies(32)[0], False)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_PAGE_RANGE


def test_slots_and_caches_past_32_bit_offsets():
    """A cache of more than 2^32 bytes and 2^31 halves: rows at its far end."""
    R, P, BS = 512, 64, 128
    pages = (1 << 31) // (BS * (R + P)) + 40
    cache = torch.zeros((pages, BS, R + P), dtype=torch.float16, device=DEV)
    g = gen(6)
    c, k = normal((5, R), g), normal((5, P), g)
    slots = i32([pages * BS - 1, pages * BS - 200, 0, pages * BS - 129, 5])
    pos = i32([1, 2, 3, 4, 5])
    f, _ = pgd.rope_frequencies(P)
    pgd.paged_latent_write(cache, None, None, c, k, slots, pos, f)
    torch.cuda.synchronize()
    lines = cache.view(-1, R + P)
    assert torch.equal(lines[slots.long(), :R], c)
    ref, tol = turned(k[:, None], pos, f, False)
    assert_turned(lines[slots.long()][:, None, R:], ref, tol)


def test_captured_and_on_another_stream():
    w = GqaRows(64, 8, 2, 128, 16, seed=8)
    f, _ = pgd.rope_frequencies(128)
    side = torch.cuda.Stream()
    b = w.before()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pgd.paged_rope_write(w.kc, w.vc, w.q_out, w.q, w.k, w.v, w.slots, w.pos, f)
    w.pos.add_(3)
    w.q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    w.check(f, False, before=b)
    side.wait_stream(torch.cuda.current_stream())
    w.pos.add_(5)
    torch.cuda.synchronize()
    pgd.paged_rope_write(w.kc, w.vc, w.q_out, w.q, w.k, w.v, w.slots, w.pos, f, stream=side)
    side.synchronize()
    w.check(f, False, before=b)
