"""Packed prompts with expanded keys and values (packed_latent_prefill) against the plain
64-bit form."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from latent_util import assert_attention, attention

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


class Prompts:
    def __init__(self, lens, H, D=128, P=64, seed=0, between=0, behind=0):
        """`between`: rows that belong to no prompt in front of the first one, NaN."""
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.H, self.D, self.P = lens, H, D, P
        self.first = between
        T = between + sum(lens) + behind
        self.T = T
        self.q = torch.randn((T, H, D + P), generator=g, device=DEV).half()
        self.kv = torch.randn((T, H, 2 * D), generator=g, device=DEV).half()
        self.down = torch.randn((T, 128 + P), generator=g, device=DEV).half()
        for x in (self.q, self.kv, self.down):
            x[:between] = float("nan")
            x[between + sum(lens):] = float("nan")
        self.k, self.v, self.k_rope = self.kv[..., :D], self.kv[..., D:], self.down[:, 128:]
        self.cu = torch.as_tensor(between + np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32,
                                  device=DEV)
        self.scale = (D + P) ** -0.5

    def run(self, dtype=torch.float16, max_len=None, **kw):
        out = torch.full((self.T, self.H, self.D), float("nan"), dtype=dtype, device=DEV)
        pgd.packed_latent_prefill(out, self.q, self.k, self.k_rope, self.v, self.cu, self.scale,
                                  max(self.lens) if max_len is None else max_len, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, what="", prompts=None, heads=None):
        r0 = self.first
        for s, n in enumerate(self.lens):
            rows = slice(r0, r0 + n)
            r0 += n
            if n == 0 or (prompts is not None and s not in prompts):
                continue
            hs = list(range(self.H)) if heads is None else heads
            k = torch.cat([self.k[rows][:, hs], self.k_rope[rows][:, None].expand(n, len(hs), self.P)], -1)
            ref, A = attention(self.q[rows][:, hs], k, self.v[rows][:, hs],
                               np.tril(np.ones((n, n), dtype=bool)), self.scale)
            vmax = float(self.v[rows].abs().max())
            assert_attention(out[rows][:, hs], ref, A, n, self.D + self.P, vmax, self.scale,
                             f"{what} prompt {s}")
        inside = torch.zeros(self.T, dtype=torch.bool, device=DEV)
        inside[self.first:self.first + sum(self.lens)] = True
        assert torch.isnan(out[~inside]).all(), "rows of no prompt were written"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [32, 64])
@pytest.mark.parametrize("H", [1, 3, 16])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_shapes(D, P, H, dtype):
    w = Prompts([1, 0, 5, 127, 128, 129, 255, 256, 257, 600, 17], H, D, P, seed=D + P + H, between=9,
                behind=70)
    w.check(w.run(dtype=dtype), f"D{D} P{P} H{H}")
    assert pgd.pgd_check_device_error() == 0


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 191, 192, 193, 383, 384, 385, 512, 513])
def test_lengths(n):
    w = Prompts([n, n, 3], 2, 128, 64, seed=n)
    w.check(w.run(), f"n {n}")


@pytest.mark.parametrize("D", [64, 128])
def test_long_prompts(D):
    w = Prompts([3001, 40, 1500], 4, D, 64, seed=D)
    w.check(w.run(), "long", heads=[0, 3])


def test_many_prompts():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    w = Prompts(lens, 5, 64, 32, seed=2)
    out = w.run()
    w.check(out, "many", prompts=set(int(x) for x in rng.integers(0, 700, 30)))
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-6])
def test_scales(scale):
    w = Prompts([300, 17], 3, 128, 64, seed=6)
    w.scale = scale
    w.check(w.run(), f"scale {scale}")


def test_strides():
    """q [heads][rows][W], k and v tensors of their own, a contiguous rotary key."""
    g = torch.Generator(device=DEV).manual_seed(1)
    w = Prompts([200, 31], 6, 128, 32, seed=5)
    w.q = w.q.transpose(0, 1).contiguous().transpose(0, 1)
    w.k = torch.randn((231, 7, 136), generator=g, device=DEV).half()[:, 1:, 8:]
    w.v = torch.randn((6, 231, 128), generator=g, device=DEV).half().transpose(0, 1)
    w.k_rope = w.k_rope.contiguous()
    w.check(w.run(), "strides")


def test_rows_of_nan_and_neighbours():
    """A query row of NaN gives NaN there alone; a neighbour prompt of NaN touches nobody."""
    w = Prompts([130, 77, 300], 2, 128, 64, seed=8)
    w.q[40, 1, 150] = float("nan")
    for x in (w.kv, w.down, w.q):
        x[130:207] = float("nan")
    out = w.run(dtype=torch.float32)
    assert torch.isnan(out[40, 1]).all() and torch.isnan(out[130:207]).all()
    ok = torch.ones((507, 2), dtype=torch.bool, device=DEV)
    ok[40, 1] = False
    ok[130:207] = False
    assert torch.isfinite(out[ok]).all()
    w.check(out, "behind NaN", prompts={2})


def test_lengths_past_the_bound_are_flagged():
    w = Prompts([100, 300, 50], 2, 64, 64, seed=9)
    good = w.run()
    out = w.run(max_len=200)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_QUERY_LEN
    assert torch.isnan(out[100:400]).all()
    assert torch.equal(out[:100], good[:100]) and torch.equal(out[400:], good[400:])
    w.cu = torch.tensor([0, 100, 90, 500], dtype=torch.int32, device=DEV)   # negative, past the end
    out = w.run(max_len=450)
    assert pgd.pgd_check_device_error() == pgd.DEVERR_QUERY_LEN
    assert torch.equal(out[:100], good[:100]) and torch.isnan(out[100:]).all()


def test_maxima_that_move():
    w = Prompts([900], 2, 128, 64, seed=10)
    w.k.mul_(torch.linspace(0.1, 2.5, 900, device=DEV)[:, None, None].half())
    out = w.run(dtype=torch.float32)
    n = 900
    k = torch.cat([w.k, w.k_rope[:, None].expand(n, 2, 64)], -1)
    ref, A = attention(w.q, k, w.v, np.tril(np.ones((n, n), dtype=bool)), w.scale)
    # |dz| <= 2^-23 W sum_d |q_d k_d| scale, as the values are not N(0, 1)
    width = max((w.q[:, h].double().abs() @ k[:, h].double().abs().T).max().item() for h in (0, 1))
    tol = (2 * 192 * 2.0 ** -23 * width * w.scale + 2.0 ** -10 + 2.0 ** -17) * A + 1e-4
    assert (np.abs(out.cpu().numpy() - ref) <= tol).all()


def test_workspace_streams_and_graphs():
    w = Prompts([700, 129, 5], 8, 128, 64, seed=11)
    ref = w.run(dtype=torch.float32)
    w.check(ref, "library scratch", heads=[0, 7])
    need = pgd.pgd_latent_prefill_plan(3, 834, 8, 128, 64)
    ws = torch.full((max(256, need),), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(w.run(dtype=torch.float32, workspace=ws), ref)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert torch.equal(w.run(dtype=torch.float32, stream=side), ref)
    graphs, outs = [], []
    for i in range(2):
        outs.append(torch.empty_like(ref))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            pgd.packed_latent_prefill(outs[i], w.q, w.k, w.k_rope, w.v, w.cu, w.scale, 700)
    for _ in range(10):
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    if need:
        with pytest.raises(pgd.PGDError, match="PGD_ERR_WORKSPACE"):
            w.run(workspace=ws[:need - 256])
