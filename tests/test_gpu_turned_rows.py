"""Turned keys as rows, which the prompt operators take, from the writes: as further query heads
of paged_rope_write, and as the one query head of a paged_latent_write that writes nothing; then
the prompts' attention over them."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
import step_util
from latent_util import LatentCase, assert_attention, attention, turned

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert pgd.pgd_check_device_error() == 0


def step(lens, BS, padding, g):
    """Slots in shuffled pages, positions and offsets of whole prompts, padding behind them."""
    n = sum(lens)
    pages = -(-n // BS)
    slots = torch.full((n + padding,), -1, dtype=torch.int32, device=DEV)
    slots[:n] = torch.randperm(pages * BS, generator=g, device=DEV)[:n].to(torch.int32)
    pos = torch.full((n + padding,), -1, dtype=torch.int32, device=DEV)
    pos[:n] = torch.as_tensor(np.concatenate([np.arange(x) for x in lens]), dtype=torch.int32)
    cu = torch.as_tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    return pages, slots, pos, cu


def test_prompts_with_rotary_positions():
    """paged_rope_write with the key heads among the queries -> packed_gqa_prefill."""
    lens, Hq, Hkv, D, BS, pad = [70, 1, 300], 8, 2, 128, 16, 4
    g = torch.Generator(device=DEV).manual_seed(1)
    pages, slots, pos, cu = step(lens, BS, pad, g)
    n = sum(lens)
    qkv = torch.randn((n + pad, Hq + 2 * Hkv, D), generator=g, device=DEV).half()
    f, _ = pgd.rope_frequencies(D, base=500000.0)
    kc, vc = (torch.zeros((pages, Hkv, BS, D), dtype=torch.float16, device=DEV) for _ in "kv")
    both = torch.full((n + pad, Hq + Hkv, D), float("nan"), dtype=torch.float16, device=DEV)
    pgd.paged_rope_write(kc, vc, both, qkv[:, :Hq + Hkv], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], slots,
                         pos, f)
    q, k, v = both[:, :Hq], both[:, Hq:], qkv[:, Hq + Hkv:]
    out = torch.full((n + pad, Hq, D), float("nan"), device=DEV)
    pgd.packed_gqa_prefill(out, q, k, v, cu, D ** -0.5, max(lens))
    torch.cuda.synchronize()
    assert torch.equal(kc.transpose(1, 2).reshape(-1, Hkv, D)[slots[:n].long()], k[:n])
    want, tol = turned(qkv[:, :Hq + Hkv], pos, f, False)
    assert ((both[:n].double() - want[:n]).abs() <= tol[:n]).all()
    assert torch.isnan(both[n:]).all() and torch.isnan(out[n:]).all()
    for s, L in enumerate(lens):
        a = int(cu[s])
        ref, A = step_util.attention(q[a:a + L], k[a:a + L], v[a:a + L], np.tril(np.ones((L, L), dtype=bool)),
                                     D ** -0.5)
        step_util.assert_attention(out[a:a + L], ref, A, L, D, float(v[a:a + L].abs().max()), f"prompt {s}")


@pytest.mark.parametrize("interleaved", [False, True])
def test_latent_prompts(interleaved):
    """paged_latent_write for the cache and the queries, and once more, without a slot, for the
    shared key -> packed_latent_prefill."""
    lens, H, D, P, R, BS, pad = [70, 1, 300], 6, 64, 32, 128, 16, 4
    g = torch.Generator(device=DEV).manual_seed(2)
    pages, slots, pos, cu = step(lens, BS, pad, g)
    n = sum(lens)
    down = torch.randn((n + pad, R + P), generator=g, device=DEV).half()
    kv = torch.randn((n + pad, H, 2 * D), generator=g, device=DEV).half()
    q = torch.randn((n + pad, H, D + P), generator=g, device=DEV).half()
    f, _ = pgd.rope_frequencies(P)
    cache = torch.zeros((pages, BS, R + P), dtype=torch.float16, device=DEV)
    pgd.paged_latent_write(cache, q[..., D:], q[..., D:], down[:, :R], down[:, R:], slots, pos, f,
                           interleaved=interleaved)
    before = cache.clone()
    key = torch.full((n + pad, P), float("nan"), dtype=torch.float16, device=DEV)
    pgd.paged_latent_write(cache, key[:, None], down[:, None, R:], down[:, :R], down[:, R:],
                           torch.full_like(slots, -1), pos, f, interleaved=interleaved)
    out = torch.full((n + pad, H, D), float("nan"), device=DEV)
    pgd.packed_latent_prefill(out, q, kv[..., :D], key, kv[..., D:], cu, (D + P) ** -0.5, max(lens))
    torch.cuda.synchronize()
    assert torch.equal(cache, before)
    assert torch.equal(cache.view(-1, R + P)[slots[:n].long(), R:], key[:n])
    assert torch.isnan(key[n:]).all() and torch.isnan(out[n:]).all()
    for s, L in enumerate(lens):
        a = slice(int(cu[s]), int(cu[s]) + L)
        k = torch.cat([kv[a, :, :D], key[a][:, None].expand(L, H, P)], -1)
        v = kv[a, :, D:]
        ref, A = attention(q[a], k, v, np.tril(np.ones((L, L), dtype=bool)), (D + P) ** -0.5)
        assert_attention(out[a], ref, A, L, D + P, float(v.abs().max()), (D + P) ** -0.5, f"prompt {s}")


@pytest.mark.parametrize("H", [129, 192, 300])
def test_heads_in_odd_numbers_of_blocks(H):
    """Three and five blocks of 64 heads a row: tiles that hold the end of one row and the start
    of the next, and a last tile with one block."""
    w = LatentCase([1, 300, 9, 2000], [1, 3, 2, 1], H, 128, 32, 16, seed=H)
    w.check(w.run(), f"H{H}")
    w = LatentCase([5000, 40], [1, 1], H, 512, 64, 64, seed=H)
    w.check(w.run(dtype=torch.float32, single=True), f"single H{H}")
