"""Refusals of the rotary and latent entry points (paged_rope_write, pgd_rope_frequencies,
paged_latent_write, paged_latent_attention, packed_latent_prefill), with the documented
status, before anything reaches a GPU, and the frequencies' closed forms."""
import ctypes
import math

import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = ctypes.c_void_p(1 << 20)        # aligned, never used: the calls are refused
B = ctypes.c_void_p(1 << 21)
NULL = ctypes.c_void_p(0)
ODD = ctypes.c_void_p((1 << 20) + 2)
EIGHT = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    return pgd.load_library()


def replaced(ptrs, **at):
    out = list(ptrs)
    for i, p in at.items():
        out[int(i[1:])] = p
    return tuple(out)


def refused(lib, got, status):
    assert got == status
    assert lib.pgd_last_error().decode() != ""


# k_cache, v_cache, q_out, q, k_new, v_new, slots, positions, inv_freq
ROPE = (A, A, B, A, A, A, A, A, A)


def rope(lib, ptrs=ROPE, magnitude=1.0, N=4, Hq=16, Hkv=4, D=128, rot=64, BS=16, NB=64,
         cache=(4 * 16 * 128, 16 * 128, 128), qo=(16 * 128, 128), q=(24 * 128, 128),
         k=(24 * 128, 128), v=(24 * 128, 128)):
    return lib.paged_rope_write(*ptrs, ctypes.c_float(magnitude), 0, N, Hq, Hkv, D, rot, BS, NB,
                                *cache, *qo, *q, *k, *v, NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hkv=0), INVALID), (dict(NB=0), INVALID),
    (dict(N=1 << 30), UNSUPPORTED), (dict(Hq=65537), UNSUPPORTED), (dict(Hkv=65537), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED), (dict(BS=4), UNSUPPORTED), (dict(rot=0), INVALID),
    (dict(rot=8), INVALID), (dict(rot=72), INVALID), (dict(rot=144), INVALID),
    (dict(magnitude=math.nan), INVALID), (dict(magnitude=math.inf), INVALID),
    (dict(cache=(4 * 16 * 128, 16 * 128, 120)), INVALID),
    (dict(cache=(4 * 16 * 128 + 4, 16 * 128, 128)), INVALID),
    (dict(qo=(16 * 128 + 4, 128)), INVALID), (dict(q=(0, 128)), INVALID),
    (dict(k=(24 * 128, -8)), INVALID), (dict(v=(1 << 39, 128)), INVALID),
    (dict(ptrs=replaced(ROPE, _0=NULL)), INVALID), (dict(ptrs=replaced(ROPE, _1=NULL)), INVALID),
    (dict(ptrs=replaced(ROPE, _2=NULL)), INVALID), (dict(ptrs=replaced(ROPE, _3=NULL)), INVALID),
    (dict(ptrs=replaced(ROPE, _4=NULL)), INVALID), (dict(ptrs=replaced(ROPE, _5=NULL)), INVALID),
    (dict(ptrs=replaced(ROPE, _6=NULL)), INVALID), (dict(ptrs=replaced(ROPE, _7=NULL)), INVALID),
    (dict(ptrs=replaced(ROPE, _8=NULL)), INVALID), (dict(ptrs=replaced(ROPE, _4=EIGHT)), INVALID),
    (dict(ptrs=replaced(ROPE, _2=EIGHT)), INVALID), (dict(ptrs=replaced(ROPE, _7=ODD)), INVALID),
    (dict(ptrs=replaced(ROPE, _8=ODD)), INVALID),
    (dict(ptrs=replaced(ROPE, _2=A)), INVALID),       # q itself, with other strides
    (dict(ptrs=replaced(ROPE, _2=A), q=(16 * 128, 256)), INVALID),
])
def test_rope_refusals(lib, kw, status):
    refused(lib, rope(lib, **kw), status)


def test_rope_of_no_rows_needs_no_arrays(lib):
    assert rope(lib, N=0, ptrs=(NULL,) * 9) == OK
    assert rope(lib, N=0, Hq=0, ptrs=(NULL,) * 9, q=(0, 0), qo=(0, 0)) == OK


# cache, q_out, q_rope, latent, k_rope, slots, positions, inv_freq
LATENT = (A, B, A, A, A, A, A, A)


def latent(lib, ptrs=LATENT, magnitude=1.0, N=4, H=16, R=512, P=64, BS=16, NB=64,
           cache=(16 * 576, 576), qo=(16 * 64, 64), q=(16 * 192, 192), c=576, k=576):
    return lib.paged_latent_write(*ptrs, ctypes.c_float(magnitude), 0, N, H, R, P, BS, NB, *cache,
                                  *qo, *q, c, k, NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INVALID), (dict(H=-1), INVALID), (dict(NB=0), INVALID), (dict(N=1 << 30), UNSUPPORTED),
    (dict(H=65537), UNSUPPORTED), (dict(R=384), UNSUPPORTED), (dict(P=16), UNSUPPORTED),
    (dict(P=128), UNSUPPORTED), (dict(BS=12), UNSUPPORTED), (dict(magnitude=math.inf), INVALID),
    (dict(cache=(16 * 576, 568)), INVALID), (dict(cache=(16 * 576 + 4, 576)), INVALID),
    (dict(cache=(0, 576)), INVALID), (dict(cache=(16 * 576, 1 << 39)), INVALID),
    (dict(c=572), INVALID), (dict(k=0), INVALID), (dict(q=(-8, 64)), INVALID),
    (dict(qo=(16 * 64, 4)), INVALID),
] + [(dict(ptrs=replaced(LATENT, **{f"_{i}": NULL})), INVALID) for i in range(8)]
  + [(dict(ptrs=replaced(LATENT, **{f"_{i}": EIGHT})), INVALID) for i in range(5)]
  + [(dict(ptrs=replaced(LATENT, **{f"_{i}": ODD})), INVALID) for i in range(5, 8)])
def test_latent_write_refusals(lib, kw, status):
    refused(lib, latent(lib, **kw), status)


def test_latent_write_of_no_rows_needs_no_arrays(lib):
    assert latent(lib, N=0, ptrs=(NULL,) * 8) == OK


# out, q, q_rope, cu_seqlens_q, cache, block_tables, seq_lens
ATTENTION = (A,) * 7


def attention(lib, ptrs=ATTENTION, out_type=1, scale=0.07, S=4, T=10, max_q=4, H=16, R=512, P=64,
              BS=16, MB=64, NB=1024, cache=(16 * 576, 576), q=(16 * 576, 576), r=(16 * 576, 576),
              ws=NULL, ws_bytes=0):
    out, qq, qr, cu, c, bt, sl = ptrs
    return lib.paged_latent_attention(out, out_type, qq, qr, cu, c, bt, sl, ctypes.c_float(scale), S,
                                      T, max_q, H, R, P, BS, MB, NB, *cache, *q, *r, ws, ws_bytes,
                                      NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(out_type=2), INVALID), (dict(out_type=-1), INVALID), (dict(S=-1), INVALID),
    (dict(T=-1), INVALID), (dict(max_q=-1), INVALID), (dict(max_q=0), INVALID), (dict(H=0), INVALID),
    (dict(H=65537), UNSUPPORTED), (dict(R=64), UNSUPPORTED), (dict(R=576), UNSUPPORTED),
    (dict(P=48), UNSUPPORTED), (dict(BS=256), UNSUPPORTED), (dict(MB=0), INVALID), (dict(NB=0), INVALID),
    (dict(MB=1 << 27), UNSUPPORTED), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(cache=(16 * 576, 568)), INVALID), (dict(cache=(16 * 576 + 2, 576)), INVALID),
    (dict(q=(16 * 576, 0)), INVALID), (dict(r=(4, 576)), INVALID), (dict(q=(1 << 39, 576)), INVALID),
    (dict(ptrs=replaced(ATTENTION, _3=NULL)), INVALID),       # a row a sequence, but 10 rows of 4
])
def test_latent_attention_sizes_refused(lib, kw, status):
    refused(lib, attention(lib, **kw), status)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the plan needs a device: with one, the "
                    "refusals behind it are the GPU test's")
def test_latent_attention_reports_a_missing_device(lib):
    assert attention(lib) == 4
    with pytest.raises(pgd.PGDError):
        pgd.pgd_latent_plan(4, 10, 4, 16, 512, 64, 16, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("kw,status",
                         [(dict(ptrs=replaced(ATTENTION, **{f"_{i}": NULL})), INVALID)
                          for i in (0, 1, 2, 4, 5, 6)]
                         + [(dict(ptrs=replaced(ATTENTION, **{f"_{i}": EIGHT})), INVALID)
                            for i in (0, 1, 2, 4)]
                         + [(dict(ptrs=replaced(ATTENTION, **{f"_{i}": ODD})), INVALID)
                            for i in (3, 5, 6)]
                         + [(dict(ws=A, ws_bytes=256), WORKSPACE),
                            (dict(ws=ctypes.c_void_p((1 << 20) + 128), ws_bytes=1 << 40), WORKSPACE),
                            (dict(S=1 << 20, T=1 << 20, max_q=1 << 20, MB=1 << 16, BS=128), UNSUPPORTED),
                            (dict(S=(1 << 31) - 1, T=(1 << 31) - 1, max_q=(1 << 31) - 1, H=65536,
                                  MB=1 << 23, BS=128), UNSUPPORTED)])
def test_latent_attention_refusals_behind_the_plan(lib, kw, status):
    refused(lib, attention(lib, **kw), status)


@pytest.mark.gpu
def test_latent_attention_counts_its_work_in_32_bits(lib):
    """Units of one sequence of 2^30 tokens: 2^23 stages each, with four times as many
    (a stage and a unit's start and end) below 2^31."""
    assert lib.pgd_latent_plan(63, 63, 1, 16, 512, 64, 128, 1 << 23, None) == OK
    refused(lib, lib.pgd_latent_plan(64, 64, 1, 16, 512, 64, 128, 1 << 23, None), UNSUPPORTED)


@pytest.mark.gpu
def test_latent_attention_of_nothing_needs_no_arrays(lib):
    assert attention(lib, S=0, ptrs=(NULL,) * 3 + (A,) + (NULL,) * 3) == OK
    assert attention(lib, T=0, ptrs=(NULL,) * 3 + (A,) + (NULL,) * 3) == OK
    assert pgd.pgd_latent_plan(4, 0, 0, 16, 512, 64, 16, 64) == 0
    assert pgd.pgd_latent_plan(0, 0, 0, 16, 512, 64, 16, 64) == 0


# out, q, k, k_rope, v, cu_seqlens
PROMPTS = (A,) * 6


def prompts(lib, ptrs=PROMPTS, out_type=1, scale=0.07, S=2, T=40, max_len=30, H=16, D=128, P=64,
            q=(16 * 192, 192), k=(16 * 256, 256), kr=576, v=(16 * 256, 256), ws=NULL, ws_bytes=0):
    out, qq, kk, kkr, vv, cu = ptrs
    return lib.packed_latent_prefill(out, out_type, qq, kk, kkr, vv, cu, ctypes.c_float(scale), S, T,
                                     max_len, H, D, P, *q, *k, kr, *v, ws, ws_bytes, NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(out_type=3), INVALID), (dict(S=-1), INVALID), (dict(T=-1), INVALID),
    (dict(max_len=-1), INVALID), (dict(H=0), INVALID), (dict(H=65537), UNSUPPORTED),
    (dict(D=256), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(P=128), UNSUPPORTED),
    (dict(scale=math.nan), INVALID), (dict(scale=-math.inf), INVALID), (dict(q=(16 * 192 + 4, 192)), INVALID),
    (dict(k=(16 * 256, 0)), INVALID), (dict(kr=-8), INVALID), (dict(v=(1 << 39, 256)), INVALID),
    (dict(T=(1 << 31) - 1, H=1024), UNSUPPORTED), (dict(ws=A, ws_bytes=256), WORKSPACE),
    (dict(ws=ctypes.c_void_p((1 << 20) + 128), ws_bytes=1 << 20), WORKSPACE),
] + [(dict(ptrs=replaced(PROMPTS, **{f"_{i}": NULL})), INVALID) for i in range(6)]
  + [(dict(ptrs=replaced(PROMPTS, **{f"_{i}": EIGHT})), INVALID) for i in range(5)]
  + [(dict(ptrs=replaced(PROMPTS, _5=ODD)), INVALID)])
def test_latent_prefill_refusals(lib, kw, status):
    refused(lib, prompts(lib, **kw), status)


def test_latent_prefill_of_nothing_needs_no_arrays(lib):
    assert prompts(lib, T=0, ptrs=(NULL,) * 6) == OK
    assert prompts(lib, S=0, ptrs=(NULL,) * 6) == OK


def test_latent_prefill_plan_closed_form():
    """16 bytes per unit (a pair of 128-token tiles of a head; one begun per prompt)
    behind 256 bytes, regions rounded up to 256."""
    assert pgd.pgd_latent_prefill_plan(4, 8192, 32, 128, 64) == 256 + (8192 // 256 + 4) * 32 * 16
    assert pgd.pgd_latent_prefill_plan(1, 1, 1, 64, 32) == 512
    assert pgd.pgd_latent_prefill_plan(3, 0, 16, 128, 64) == 0
    with pytest.raises(pgd.PGDError):
        pgd.pgd_latent_prefill_plan(3, 100, 16, 256, 64)


# ---------------------------------------------------------------- frequencies
def table(*a, **kw):
    f, magnitude = pgd.rope_frequencies(*a, device="cpu", **kw)
    return f.double(), magnitude


def close(got, want):
    """Rounded once to fp32."""
    want = torch.as_tensor(want, dtype=torch.float64)
    assert ((got - want).abs() <= 2.0 ** -24 * want.abs() * (1 + 1e-9)).all(), (got, want)


@pytest.mark.parametrize("rot,base", [(4, 10000.0), (64, 10000.0), (128, 500000.0), (256, 1e6), (34, 2.5)])
def test_frequencies_plain_and_linear(rot, base):
    want = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    f, m = table(rot, base)
    assert f.numel() == rot // 2 and m == 1.0
    close(f, want)
    f, m = table(rot, base, scaling="linear", factor=8.0)
    assert m == 1.0
    close(f, [x / 8.0 for x in want])


def test_frequencies_base():
    rot, factor = 64, 4.0
    f, m = table(rot, scaling="base", factor=factor)
    plain = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    assert m == 1.0 and f[0] == 1.0
    close(f, [(10000.0 * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot) for i in range(rot // 2)])
    assert abs(f[-1] / (plain[-1] / factor) - 1) < 1e-6      # the lowest shrinks by the factor
    close(table(rot, scaling="base", factor=1.0)[0], plain)


def test_frequencies_by_parts():
    """Pair i turns original_len f_i / 2 pi times in the trained context: fast ones stay,
    slow ones shrink by the factor, and in between it goes by the index."""
    rot, base, factor, length, fast, slow = 64, 10000.0, 40.0, 4096.0, 32.0, 1.0
    f, m = table(rot, base, scaling="by_parts", factor=factor, original_len=length, beta_fast=fast,
                 beta_slow=slow)
    assert abs(m - (0.1 * math.log(factor) + 1.0)) < 1e-7
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    turns = [length * x / (2 * math.pi) for x in plain]
    low = math.floor(rot * math.log(length / (fast * 2 * math.pi)) / (2 * math.log(base)))
    high = math.ceil(rot * math.log(length / (slow * 2 * math.pi)) / (2 * math.log(base)))
    for i, x in enumerate(plain):
        part = min(max((i - low) / (high - low), 0.0), 1.0)
        close(f[i:i + 1], [x * (1 - part) + x / factor * part])
        if turns[i] > fast * base ** (2.0 / rot):
            assert part == 0.0
        if turns[i] < slow / base ** (2.0 / rot):
            assert part == 1.0
    close(table(rot, base, scaling="by_parts", factor=1.0, original_len=length)[0], plain)
    # a context in which no pair turns often enough: all but the first shrink
    f, _ = table(rot, base, scaling="by_parts", factor=2.0, original_len=1.0)
    close(f, plain[:1] + [x / 2 for x in plain[1:]])


@pytest.mark.parametrize("args", [
    (3, 1e4, 0, 1.0, 0, 32, 1), (2, 1e4, 0, 1.0, 0, 32, 1), (65538, 1e4, 0, 1.0, 0, 32, 1),
    (64, 1.0, 0, 1.0, 0, 32, 1), (64, math.nan, 0, 1.0, 0, 32, 1), (64, math.inf, 0, 1.0, 0, 32, 1),
    (64, 1e4, 4, 1.0, 0, 32, 1), (64, 1e4, -1, 1.0, 0, 32, 1), (64, 1e4, 1, 0.5, 0, 32, 1),
    (64, 1e4, 2, math.nan, 0, 32, 1), (64, 1e4, 3, 4.0, 0, 32, 1), (64, 1e4, 3, 4.0, 4096, 1, 1),
    (64, 1e4, 3, 4.0, 4096, 32, 0), (64, 1e4, 3, math.inf, 4096, 32, 1), (64, 1e4, 3, 4.0, math.nan, 32, 1),
])
def test_frequencies_refusals(lib, args):
    rot, base, scaling, *rest = args
    out = (ctypes.c_float * 32768)()
    got = lib.pgd_rope_frequencies(ctypes.cast(out, ctypes.c_void_p), None, rot, base, scaling, *rest)
    refused(lib, got, INVALID)
    assert all(x == 0.0 for x in out[:64])
    refused(lib, lib.pgd_rope_frequencies(None, None, 64, 1e4, 0, 1.0, 0.0, 32.0, 1.0), INVALID)


def test_frequencies_by_name():
    with pytest.raises(ValueError, match="linear"):
        pgd.rope_frequencies(64, scaling="Linear", device="cpu")
    with pytest.raises(pgd.PGDError):
        pgd.rope_frequencies(0, device="cpu")


# ---------------------------------------------------------------- binding
def test_binding_refusals():
    i = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(32)
    q = torch.zeros((4, 8, 128), dtype=torch.float16)
    k = torch.zeros((2, 8, 16, 128), dtype=torch.float16)
    c = torch.zeros((2, 16, 576), dtype=torch.float16)
    with pytest.raises((TypeError, ValueError), match="CUDA"):
        pgd.paged_rope_write(k, k, q, q, q, q, i, i, f)
    with pytest.raises((TypeError, ValueError), match="CUDA"):
        pgd.paged_latent_write(c, q, q, q[:, 0], q[:, 1], i, i, f)
    with pytest.raises((TypeError, ValueError), match="CUDA"):
        pgd.paged_latent_attention(q, q, q, c, i.view(4, 1), i, 0.1)
    with pytest.raises((TypeError, ValueError), match="CUDA"):
        pgd.packed_latent_prefill(q, q, q, q[:, 0], q, i, 0.1, 4)


@pytest.mark.gpu
def test_binding_refuses_shapes_types_and_devices_by_name():
    dev = "cuda:0"
    i = torch.zeros(4, dtype=torch.int32, device=dev)
    f = torch.zeros(32, device=dev)
    q = torch.zeros((4, 8, 128), dtype=torch.float16, device=dev)
    k = torch.zeros((2, 8, 16, 128), dtype=torch.float16, device=dev)

    def rope(*bad, **at):
        a = dict(k_cache=k, v_cache=k, q_out=q, q=q, k_new=q, v_new=q, slots=i, positions=i, inv_freq=f)
        a.update(at)
        with pytest.raises(bad or (ValueError, TypeError)):
            pgd.paged_rope_write(**a)
    rope(v_new=q[:, :4])
    rope(q_out=None)
    rope(q=None)
    rope(q_out=q[:3])
    rope(q=q[..., :64])
    rope(slots=i[:3])
    rope(positions=i.long())
    rope(inv_freq=f.double())
    rope(inv_freq=f.cpu())
    rope(inv_freq=[0.1] * 32)
    rope(k_cache=k[:, :4])
    rope(v_cache=k.float())
    rope(slots=i.cpu())
    rope(k_new=q.float())
    rope(k_new=None)
    rope(layout=(4, 16, 2, (8 * 16 * 128, 16 * 128, 128)))
    rope(pgd.PGDError, inv_freq=f[:12])                     # 24 of 128: not a multiple of 16
    rope(pgd.PGDError, inv_freq=torch.zeros(72, device=dev))

    c = torch.zeros((2, 16, 576), dtype=torch.float16, device=dev)
    lat = torch.zeros((4, 512), dtype=torch.float16, device=dev)
    kr = torch.zeros((4, 64), dtype=torch.float16, device=dev)
    qr = torch.zeros((4, 8, 64), dtype=torch.float16, device=dev)

    def write(*bad, **at):
        a = dict(cache=c, q_out=qr, q_rope=qr, latent=lat, k_rope=kr, slots=i, positions=i, inv_freq=f)
        a.update(at)
        with pytest.raises(bad or (ValueError, TypeError)):
            pgd.paged_latent_write(**a)
    write(cache=c[..., :512])
    write(cache=c.float())
    write(cache=None)
    write(cache=c.transpose(1, 2))
    write(q_out=None)
    write(q_out=qr[:, :4])
    write(q_rope=qr[..., :32])
    write(latent=lat[:3])
    write(latent=lat.cpu())
    write(k_rope=kr.t())
    write(inv_freq=f[:16])
    write(positions=i[:2])
    write(slots=None)

    qa = torch.zeros((4, 8, 512), dtype=torch.float16, device=dev)

    def attend(*bad, **at):
        a = dict(out=qa.clone(), q=qa, q_rope=qr, cache=c, block_tables=i.view(4, 1), seq_lens=i, scale=0.1)
        a.update(at)
        with pytest.raises(bad or (ValueError, TypeError)):
            pgd.paged_latent_attention(**a)
    attend(out=qa.double())
    attend(out=qa[:3])
    attend(out=qa.transpose(0, 1))
    attend(q_rope=qr[:, :4])
    attend(q_rope=None)
    attend(cache=c[..., :512])
    attend(cache=c.cpu())
    attend(block_tables=i.view(4, 1).long())
    attend(block_tables=i)
    attend(seq_lens=i[:3])
    attend(cu_seqlens_q=i)                                    # S + 1 values
    attend(cu_seqlens_q=[0, 1, 2, 3, 4])
    attend(block_tables=i[:2].view(2, 1), seq_lens=i[:2])     # 4 rows of 2 sequences
    attend(workspace=torch.zeros(1 << 22, dtype=torch.uint8))
    attend(pgd.PGDError, workspace=torch.zeros(8, dtype=torch.uint8, device=dev))

    qe = torch.zeros((4, 8, 192), dtype=torch.float16, device=dev)

    def prefill(*bad, **at):
        a = dict(out=q.clone(), q=qe, k=q, k_rope=kr, v=q, cu_seqlens=i, scale=0.1, max_len=4)
        a.update(at)
        with pytest.raises(bad or (ValueError, TypeError)):
            pgd.packed_latent_prefill(**a)
    prefill(q=q)
    prefill(k=q[:, :4])
    prefill(k_rope=kr[:3])
    prefill(k_rope=qr)
    prefill(v=q[:3])
    prefill(out=q[..., :64])
    prefill(cu_seqlens=i[:0])
    prefill(cu_seqlens=i.float())
    prefill(cu_seqlens=None)
    prefill(v=q.cpu())
    prefill(pgd.PGDError, max_len=-1)
