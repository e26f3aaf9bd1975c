"""Rules of the memory model that a run of the kernels cannot show to be broken, in the
sources of the rotary and latent kernels (as test_step_sources has them for the others)."""
import re

import pytest

from test_step_sources import source


@pytest.mark.parametrize("name,inputs", [
    ("pgd_rope.cu", {"slots", "positions", "inv_freq"}),
    ("pgd_latent_prefill.cu", {"cu_seqlens"}), ("pgd_latent.cu", set()),
])
def test_non_coherent_loads_are_of_the_callers_inputs(name, inputs):
    """What a launch before may be writing while the kernel already runs is read by plain
    loads: the lists of units, the pieces, and in pgd_latent.cu, whose first kernel starts
    under the launch before the call, the caller's arrays too."""
    read = set(re.findall(r"__ldg\(\s*(?:reinterpret_cast<[^>]*>\()?p\.(\w+)", source(name)))
    assert read <= inputs, read - inputs
    if name == "pgd_latent.cu":
        assert "ldg" not in source(name) and "ld.global.nc" not in source(name)


def test_nothing_is_read_in_front_of_the_wait():
    """The latent kernel sets itself up before griddep_wait without a look at global memory
    (but for the tensor maps, which are parameters), and so does the joining kernel."""
    text = source("pgd_latent.cu")
    for kernel, behind in (("paged_latent_kernel(", "latent_seq"), ("paged_latent_join_kernel(", "p.cut")):
        body = text[text.index(kernel):]
        set_up = body[body.index("{"):body.index("griddep_wait()")]
        assert behind not in set_up
        assert not re.search(r"p\.(seq_lens|cu_q|block_tables|part_o|part_ml|cut|out|err)\b", set_up)


@pytest.mark.parametrize("name", ["pgd_latent.cu", "pgd_latent_prefill.cu"])
def test_tensor_memory_loads_are_used_behind_their_wait(name):
    parts = source(name).split("tc_wait_ld();")
    assert len(parts) > 1
    for behind in parts[1:]:
        first_use = re.search(r"tc_ld_ready\(|\*=|make_float4|tc_st32|fmax|v\[|o\[", behind)
        assert first_use and first_use.group(0) == "tc_ld_ready(", behind[:300]


@pytest.mark.parametrize("name", ["pgd_latent.cu", "pgd_latent_prefill.cu"])
def test_every_wait_is_bounded(name):
    """No wait on a barrier but with a budget of time (or the look that is repeated by one)."""
    for call in re.findall(r"mbar_\w*wait\w*|mbar_try\w*", source(name)):
        assert call.endswith("_bounded") or call.startswith("mbar_try"), call
