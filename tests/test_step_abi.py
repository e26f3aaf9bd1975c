"""Refusals of the step's entry points (paged_kv_slots, paged_kv_write,
paged_gqa_tree, packed_gqa_prefill), with the documented status, before anything reaches a GPU."""
import ctypes
import math

import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
A = ctypes.c_void_p(1 << 20)        # aligned, never used: the calls are refused
B = ctypes.c_void_p(1 << 21)
NULL = ctypes.c_void_p(0)
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    return pgd.load_library()


SLOTS = ("slots", "positions", "cu", "lens", "end", "tables", "ctx", "new", "free", "start")


def slots(lib, S=4, N=8, F=16, BS=16, MB=64, NB=1024, **ptr):
    at = {n: ctypes.c_void_p((i + 1) << 20) for i, n in enumerate(SLOTS)}
    at.update(ptr)
    return lib.paged_kv_slots(*[at[n] for n in SLOTS], S, N, F, BS, MB, NB, NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), INVALID), (dict(N=-1), INVALID), (dict(F=-1), INVALID),
    (dict(BS=12), UNSUPPORTED), (dict(MB=0), INVALID), (dict(NB=0), INVALID),
    (dict(MB=1 << 28), UNSUPPORTED), (dict(NB=(1 << 27) + 1), UNSUPPORTED),
    (dict(S=16385), UNSUPPORTED), (dict(N=1 << 30), UNSUPPORTED), (dict(F=1 << 30), UNSUPPORTED),
    (dict(slots=NULL), INVALID), (dict(cu=NULL), INVALID), (dict(lens=NULL), INVALID),
    (dict(end=NULL), INVALID), (dict(tables=NULL), INVALID), (dict(ctx=NULL), INVALID),
    (dict(new=NULL), INVALID), (dict(free=NULL), INVALID), (dict(positions=ODD), INVALID),
    (dict(start=ODD), INVALID), (dict(end=A, start=A), INVALID), (dict(lens=A, ctx=A), INVALID),
    (dict(lens=A, new=A), INVALID),
])
def test_slots_refusals(lib, kw, status):
    assert slots(lib, **kw) == status
    assert lib.pgd_last_error().decode() != ""


def write(lib, N=4, Hkv=8, D=128, BS=16, NB=64, strides=(8 * 16 * 128, 16 * 128, 128),
          src=(8 * 128, 128), ptrs=(A, A, A, A, A)):
    return lib.paged_kv_write(*ptrs, N, Hkv, D, BS, NB, *strides, *src, NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), INVALID), (dict(Hkv=0), INVALID), (dict(NB=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(BS=4), UNSUPPORTED), (dict(Hkv=65537), UNSUPPORTED),
    (dict(strides=(8 * 16 * 128, 16 * 128, 120)), INVALID),
    (dict(strides=(8 * 16 * 128 + 4, 16 * 128, 128)), INVALID),
    (dict(src=(8 * 128 + 4, 128)), INVALID), (dict(src=(8 * 128, 0)), INVALID),
    (dict(src=(-8, 128)), INVALID), (dict(src=(1 << 39, 128)), INVALID),
    (dict(ptrs=(NULL, A, A, A, A)), INVALID), (dict(ptrs=(A, A, A, A, NULL)), INVALID),
    (dict(ptrs=(A, A, ODD, A, A)), INVALID), (dict(ptrs=(A, A, A, A, ODD)), INVALID),
])
def test_write_refusals(lib, kw, status):
    assert write(lib, **kw) == status
    assert lib.pgd_last_error().decode() != ""


def test_write_of_no_rows_needs_no_arrays(lib):
    assert write(lib, N=0, ptrs=(NULL,) * 5) == 0


def tree(lib, out_type=1, T=40, max_q=16, S=4, Hq=32, Hkv=8, D=128, BS=16, MB=64, NB=1024,
         scale=0.1, strides=None, ptrs=(A,) * 8, ws=NULL, ws_bytes=0):
    strides = strides or (Hkv * BS * D, BS * D, D)
    out, q, cu, parents, k, v, bt, sl = ptrs
    return lib.paged_gqa_tree(out, out_type, q, cu, parents, k, v, bt, sl, ctypes.c_float(scale), S,
                              T, max_q, Hq, Hkv, D, BS, MB, NB, *strides, ws, ws_bytes, NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(out_type=2), INVALID), (dict(out_type=-1), INVALID), (dict(max_q=257), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED), (dict(BS=4), UNSUPPORTED), (dict(Hq=30), INVALID),
    (dict(Hq=129 * 8), UNSUPPORTED), (dict(MB=0), INVALID), (dict(T=-1), INVALID),
    (dict(T=4, max_q=0), INVALID), (dict(S=-1), INVALID), (dict(MB=1 << 28), UNSUPPORTED),
])
def test_tree_sizes_refused(lib, kw, status):
    assert tree(lib, **kw) == status
    assert lib.pgd_last_error().decode() != ""


@pytest.mark.skipif(torch.cuda.is_available(), reason="the plan needs a device: with one, the "
                    "refusals behind it are the GPU test's")
def test_tree_reports_a_missing_device(lib):
    assert tree(lib) == 4


def prefill(lib, out_type=1, S=2, T=40, max_len=30, Hq=32, Hkv=8, D=128, scale=0.1,
            strides=(48 * 128, 128) * 3, ptrs=(A,) * 5, ws=NULL, ws_bytes=0):
    out, q, k, v, cu = ptrs
    return lib.packed_gqa_prefill(out, out_type, q, k, v, cu, ctypes.c_float(scale), S, T, max_len,
                                  Hq, Hkv, D, *strides, ws, ws_bytes, NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(out_type=7), INVALID), (dict(S=-1), INVALID), (dict(T=-1), INVALID),
    (dict(max_len=-1), INVALID), (dict(Hq=30), INVALID), (dict(Hq=0), INVALID),
    (dict(Hq=129 * 8), UNSUPPORTED), (dict(Hq=1 << 17, Hkv=1 << 17), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(strides=(48 * 128 + 4, 128) + (48 * 128, 128) * 2), INVALID),
    (dict(strides=(48 * 128, 128) * 2 + (48 * 128, 0)), INVALID),
    (dict(strides=(48 * 128, 128) * 2 + (1 << 39, 128)), INVALID),
    (dict(ptrs=(NULL, A, A, A, A)), INVALID), (dict(ptrs=(A, A, A, A, NULL)), INVALID),
    (dict(ptrs=(A, ctypes.c_void_p((1 << 20) + 8), A, A, A)), INVALID),
    (dict(ptrs=(A, A, A, A, ODD)), INVALID), (dict(ws=A, ws_bytes=256), WORKSPACE),
    (dict(ws=ctypes.c_void_p((1 << 20) + 128), ws_bytes=1 << 20), WORKSPACE),
    (dict(T=(1 << 31) - 1, Hkv=4096, Hq=4096), UNSUPPORTED),
])
def test_prefill_refusals(lib, kw, status):
    assert prefill(lib, **kw) == status
    assert lib.pgd_last_error().decode() != ""


def test_prefill_of_nothing_needs_no_arrays(lib):
    assert prefill(lib, T=0, ptrs=(NULL,) * 5) == 0
    assert prefill(lib, S=0, ptrs=(NULL,) * 5) == 0


def test_prefill_plan_closed_form():
    """16 bytes per unit of 2 tiles of 128 / G tokens (one tile at head_dim 256) and KV
    head, one begun per prompt, behind 256 bytes; regions rounded up to 256."""
    assert pgd.pgd_prefill_plan(4, 8192, 32, 8, 128) == 256 + (8192 // 64 + 4) * 8 * 16
    assert pgd.pgd_prefill_plan(3, 100, 24, 4, 256) == 256 + 512
    assert pgd.pgd_prefill_plan(3, 0, 24, 4, 256) == 0
    with pytest.raises(pgd.PGDError):
        pgd.pgd_prefill_plan(3, 100, 24, 5, 256)


def test_binding_refusals():
    i = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros((4, 8, 128), dtype=torch.float16)
    k = torch.zeros((2, 8, 16, 128), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        pgd.paged_kv_slots(i, i, i, i[:1], i.view(1, 4), i, i, i, 16, 64)
    with pytest.raises(TypeError, match="float16 CUDA"):
        pgd.paged_kv_write(k, k, q, q, i)
    with pytest.raises(ValueError, match="CUDA"):
        pgd.paged_gqa_tree(q, q, i, i, k, k, i.view(1, 4), i, 0.1, 4)
    with pytest.raises(TypeError, match="float32 or float16"):
        pgd.paged_gqa_tree(q.double(), q, i, i, k, k, i.view(1, 4), i, 0.1, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pgd.packed_gqa_prefill(q, q, q, q, i, 0.1, 4)
    with pytest.raises(TypeError, match="torch.Tensor|has no|float"):
        pgd.packed_gqa_prefill(None, q, q, q, i, 0.1, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("kw,status", [
    (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(NB=0), INVALID),
    (dict(strides=(8 * 16 * 128, 16 * 128, 120)), INVALID),
    (dict(ptrs=(A, A, A, NULL, A, A, A, A)), INVALID),
    (dict(ptrs=(A, A, A, ODD, A, A, A, A)), INVALID),
    (dict(ptrs=(NULL, A, A, A, A, A, A, A)), INVALID),
    (dict(ptrs=(ctypes.c_void_p((1 << 20) + 8), A, A, A, A, A, A, A)), INVALID),
    (dict(ws=A, ws_bytes=16), WORKSPACE),
])
def test_tree_refusals_behind_the_plan(lib, kw, status):
    assert tree(lib, **kw) == status
    assert lib.pgd_last_error().decode() != ""


@pytest.mark.gpu
def test_binding_refuses_mixed_devices_and_shapes():
    dev = "cuda:0"
    i = torch.zeros(4, dtype=torch.int32, device=dev)
    q = torch.zeros((4, 8, 128), dtype=torch.float16, device=dev)
    k = torch.zeros((2, 8, 16, 128), dtype=torch.float16, device=dev)
    with pytest.raises(ValueError):
        pgd.paged_gqa_tree(q, q, i, i, k, k, i.view(4, 1), i, 0.1, 4)     # cu needs S + 1
    with pytest.raises(ValueError):
        pgd.paged_kv_write(k, k, q.transpose(1, 2), q.transpose(1, 2), i)
    with pytest.raises(ValueError):
        pgd.paged_kv_write(k, k, q[:, :4], q[:, :4], i)                   # heads of the cache
    with pytest.raises(ValueError):
        pgd.paged_kv_slots(i, i, i, i[:1], i.view(4, 1), i, i, i, 16, 64)
    with pytest.raises(ValueError, match="contiguous"):
        pgd.packed_gqa_prefill(q, q.transpose(1, 2), q, q, i, 0.1, 4)
    with pytest.raises(ValueError, match="shapes"):
        pgd.packed_gqa_prefill(q, q, q[:3], q[:3], i, 0.1, 4)
    with pytest.raises(ValueError):
        pgd.packed_gqa_prefill(q, q, q, q, i[:0], 0.1, 4)
    for bad in (i.float(), i.view(2, 2), None, [0, 1]):
        with pytest.raises((TypeError, ValueError, AttributeError)):
            pgd.packed_gqa_prefill(q, q, q, q, bad, 0.1, 4)
