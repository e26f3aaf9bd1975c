"""Rules of the memory model that a run of the kernels cannot show to be broken:
read in the sources of the step's kernels."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_gqa_decode_03_gb300", "csrc")


def source(name):
    """The file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


# what these kernels read through __ldg (ld.global.nc): memory that nothing
# writes while they run, which the caller's inputs are
INPUTS = {"cu_seqlens", "cu_q", "parents", "seq_lens", "block_tables", "context_lens",
          "query_lens", "free_start", "free_pages", "slots", "k_new", "v_new"}


@pytest.mark.parametrize("name", ["pgd_prefill.cu", "pgd_tree.cu", "pgd_kv.cu"])
def test_non_coherent_loads_are_of_the_callers_inputs(name):
    """Scratch that the launch before writes (the unit list, the pieces) while a
    kernel launched with programmatic serialization already runs is not constant
    for that kernel's lifetime, so it may not be read through ld.global.nc."""
    read = set(re.findall(r"__ldg\(\s*(?:reinterpret_cast<[^>]*>\()?p\.(\w+)", source(name)))
    assert read and read <= INPUTS, read - INPUTS


@pytest.mark.parametrize("name", ["pgd_prefill.cu", "pgd_tree.cu", "pgd_rows.cuh", "pgd_varlen.cu"])
def test_tensor_memory_loads_are_used_behind_their_wait(name):
    """tcgen05.ld is asynchronous: its registers may be read behind tcgen05.wait::ld
    only.  The wait names no register, so arithmetic on them (which is not
    volatile) may be moved in front of it unless tc_ld_ready, right behind the
    wait, ties them to that place."""
    parts = source(name).split("tc_wait_ld();")
    assert len(parts) > 1
    for behind in parts[1:]:
        first_use = re.search(r"tc_ld_ready\(|\*=|make_float4|tc_st32|fmax|x\[32", behind)
        assert first_use and first_use.group(0) == "tc_ld_ready(", behind[:300]
