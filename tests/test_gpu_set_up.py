"""The tree and prompt kernels are set up by the first call that needs them: a
set-up that fails is that call's failure alone, and a first call may be captured
into a graph.  Each in a process of its own, where nothing is set up yet."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import pytest
import torch
import paged_gqa_decode_03_gb300 as pgd
import test_gpu_prefill as prefill
import test_gpu_tree as tree
from parity_util import assert_parity, oracle_out, run
from paged_gqa_decode_03_gb300.workloads import make_workload

def decode():
    w = make_workload("tiny", device="cuda:0")
    assert_parity(run(w, P=0).cpu().numpy(), oracle_out(w), "decode")

CTX, N = [300, 40, 2000], [30, 9, 70]
D = int(sys.argv[1])
w, trees, parents = tree.case(CTX, N, 16, 4, D, 16, seed=4)
c = prefill.case([70, 300], 8, 2, D, seed=3)
"""

FAILED = HEAD + """
for call, check in ((lambda: tree.run(w, parents), lambda o: tree.check(o, w, trees, CTX, "tree")),
                    (lambda: prefill.run(c), lambda o: prefill.check(o, c, "prompts"))):
    pgd.pgd_test_fail_next_set_up()
    decode()
    with pytest.raises(pgd.PGDError, match="withheld") as e:
        call()
    assert e.value.status == 4
    decode()
    check(call())
    pgd.pgd_test_fail_next_set_up()
    check(call())                      # set up: nothing to fail
    pgd.pgd_test_fail_next_set_up(False)
    assert pgd.pgd_check_device_error() == 0
print("as it should")
"""

CAPTURED = HEAD + """
out = torch.zeros((w.total_q, w.Hq, D), dtype=torch.float16, device="cuda:0")
out2 = torch.zeros(c["q"].shape, dtype=torch.float16, device="cuda:0")
if sys.argv[2] == "after a decode":
    decode()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    pgd.paged_gqa_tree(out, w.q, w.cu_seqlens_q, parents, w.k_cache, w.v_cache, w.block_tables,
                       w.seq_lens, w.scale, w.max_q_len)
    pgd.packed_gqa_prefill(out2, c["q"], c["k"], c["v"], c["cu"], c["scale"], 300)
for _ in range(2):
    out.zero_()
    out2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    tree.check(out, w, trees, CTX, "tree")
    prefill.check(out2, c, "prompts")
assert pgd.pgd_check_device_error() == 0
print("as it should")
"""


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def own_process(code, *args):
    r = subprocess.run([sys.executable, "-c", code.format(root=ROOT), *map(str, args)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as it should" in r.stdout, r.stdout + r.stderr[-3000:]


@pytest.mark.parametrize("D", [64, 128, 256])
def test_failed_set_up_is_one_calls_failure(D):
    own_process(FAILED, D)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("when", ["first of all", "after a decode"])
def test_first_call_captured(D, when):
    own_process(CAPTURED, D, when)
