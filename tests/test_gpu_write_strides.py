"""paged_kv_write of K and V rows with different strides, the ones that
packed_gqa_prefill attends to in the same step; paged_kv_write_strided's refusals."""
import ctypes

import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd
from test_gpu_kv_step import plain_write, write_case

DEV = "cuda:0"
INVALID = 1


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hkv,N", [(1, 1), (1, 37), (3, 1), (4, 300)])
@pytest.mark.parametrize("BS,token_major", [(16, False), (32, True)])
def test_rows_of_different_strides(D, Hkv, N, BS, token_major):
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    kc, vc, slots, g = write_case(N, Hkv, D, BS, token_major, seed=N + D, skip=N // 4)
    layout = (Hkv, BS, kc.shape[0], pgd.kv_strides("token_major", Hkv, BS, D)) if token_major else None
    rows = torch.randn((2, N, Hkv, D), generator=g, device=DEV).half()
    forms = [rows[0], torch.cat([rows[0], rows[0]], 1)[:, :Hkv],              # packed, fused
             rows[0].transpose(0, 1).contiguous().transpose(0, 1),           # head-major
             torch.nn.functional.pad(rows[0], (0, 24))[:, :, :D]]            # padded rows
    for k in forms:
        for v in forms:
            assert torch.equal(k, rows[0]) and torch.equal(v, rows[0])
            k2, v2 = kc.clone(), vc.clone()
            pgd.paged_kv_write(k2, v2, k, v, slots, layout=layout)
            torch.cuda.synchronize()
            assert torch.equal(k2, plain_write(kc, rows[0], slots, BS, token_major))
            assert torch.equal(v2, plain_write(vc, rows[0], slots, BS, token_major))
    # each from its own rows
    k2, v2 = kc.clone(), vc.clone()
    pgd.paged_kv_write(k2, v2, forms[1], rows[1], slots, layout=layout)
    torch.cuda.synchronize()
    assert torch.equal(k2, plain_write(kc, rows[0], slots, BS, token_major))
    assert torch.equal(v2, plain_write(vc, rows[1], slots, BS, token_major))
    assert pgd.pgd_check_device_error() == 0


@pytest.mark.parametrize("strides", [(0, 128, 1024, 128), (1024, 4, 1024, 128),
                                     (1024, 128, 1 << 39, 128), (1024, 128, 1024, -8),
                                     (1024, 128, 1028, 128)])
def test_strides_refused(strides):
    a = ctypes.c_void_p(1 << 20)        # aligned, never used
    lib = pgd.load_library()
    assert lib.paged_kv_write_strided(a, a, a, a, a, 4, 8, 128, 16, 64, 8 * 16 * 128, 16 * 128, 128,
                                      *strides, ctypes.c_void_p(0)) == INVALID
    assert "source strides" in lib.pgd_last_error().decode()
