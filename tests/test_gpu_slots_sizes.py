"""paged_kv_slots around the request counts at which its shared memory passes
48 KB, in a process of its own: a larger call beforehand would have asked for
more shared memory on the kernel's behalf."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import numpy as np
import paged_gqa_decode_03_gb300 as pgd
import test_gpu_kv_step as t

for S in (1, 5119, 5120, 6127, 6128, 6143, 6144, 8000):
    rng = np.random.RandomState(S)
    c = t.step(rng.randint(0, 40, S), rng.randint(0, 3, S), 16, spare=5)
    t.check(c, t.run(c))
assert pgd.pgd_check_device_error() == 0
print("every count right")
"""


def test_counts_around_48_kb_of_shared_memory():
    import __graft_entry__
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", CODE.format(root=ROOT)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "every count right" in r.stdout, r.stdout + r.stderr[-3000:]
