"""What is no tensor is refused by name, with a TypeError, by the step's calls of
the binding."""
import pytest
import torch

import paged_gqa_decode_03_gb300 as pgd


def calls(dev):
    """Per call: its tensor arguments by name (in order), and the call itself."""
    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=dev)

    def f16(*shape):
        return torch.zeros(shape, dtype=torch.float16, device=dev)
    cache = dict(k_cache=f16(2, 8, 16, 128), v_cache=f16(2, 8, 16, 128))
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    return {
        "slots": (dict(slots=i32(4), cu_seqlens_q=i32(3), seq_lens=i32(2), free_end=i32(1),
                       block_tables=i32(2, 4), context_lens=i32(2), query_lens=i32(2),
                       free_pages=i32(4), free_start=i32(1), positions=i32(4)),
                  lambda a: pgd.paged_kv_slots(*list(a.values())[:8], 16, 64,
                                               free_start=a["free_start"],
                                               positions=a["positions"])),
        "write": (dict(cache, k_new=f16(4, 8, 128), v_new=f16(4, 8, 128), slots=i32(4)),
                  lambda a: pgd.paged_kv_write(*a.values())),
        "tree": (dict(out=f16(4, 8, 128), q=f16(4, 8, 128), cu_seqlens_q=i32(3), parents=i32(4),
                      **cache, block_tables=i32(2, 4), seq_lens=i32(2), workspace=ws),
                 lambda a: pgd.paged_gqa_tree(*list(a.values())[:8], 0.1, 4,
                                              workspace=a["workspace"])),
        "prefill": (dict(out=f16(4, 8, 128), q=f16(4, 8, 128), k=f16(4, 8, 128), v=f16(4, 8, 128),
                         cu_seqlens=i32(3), workspace=ws),
                    lambda a: pgd.packed_gqa_prefill(*list(a.values())[:5], 0.1, 4,
                                                     workspace=a["workspace"])),
    }


@pytest.mark.parametrize("bad", [None, [0, 1], 3])
def test_no_tensor_on_the_cpu(bad):
    slots, call = calls("cpu")["slots"]
    with pytest.raises(TypeError, match="slots must be a torch.Tensor"):
        call(dict(slots, slots=bad))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["slots", "write", "tree", "prefill"])
@pytest.mark.parametrize("bad", [None, [0, 1], 3])
def test_no_tensor(name, bad):
    args, call = calls("cuda:0")[name]
    for x in args:
        if bad is None and x in ("free_start", "positions", "workspace"):
            continue                                  # these may be left out
        with pytest.raises(TypeError, match=f"{x} must be|layout"):
            call(dict(args, **{x: bad}))
    assert pgd.pgd_check_device_error() == 0
