"""What the bench line's DRAM figure is tied to: every source that the decode kernels are made of."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "paged_kv_decode_12_gb300", "csrc")


def included(name, seen):
    """`name` and what it includes of this directory, and so on."""
    if name not in seen:
        seen.add(name)
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            for inner in re.findall(r'^#include "([^"/]+)"', f.read(), flags=re.M):
                included(inner, seen)
    return seen


def test_the_digest_covers_the_decode_kernels():
    need = included("pkv_step.cu", set())
    assert {"pkv_step.cuh", "pkv_device.cuh", "pkv_fp8.cuh"} <= need <= set(bench.KERNEL_SOURCES)
    assert all(os.path.exists(os.path.join(CSRC, name)) for name in bench.KERNEL_SOURCES)
