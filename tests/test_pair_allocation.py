"""An allocation of tensor memory for a pair of CTAs begins once both of them run: each kernel that makes one arrives at its
cluster's barrier when it starts and waits for it first.  (Where a pair starts beside other work, one CTA can be late, and an
allocation that the other one has begun by then can wait for good.  That it does is not tried; the source is read.)"""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ozaki_ii_fp64_gb300", "csrc")


def kernels():
    """(file, what a kernel does before its pair allocation), from its __global__ on."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for at in (m.start() for m in re.finditer(r"\btmem_alloc_pair\(", text)):
            found.append((os.path.basename(path), text[text.rfind("__global__", 0, at):at]))
    return found


def test_there_are_some():
    assert {name for name, _ in kernels()} == {"gemm_fp4.cu", "linear.cu", "mx.cu"}


@pytest.mark.parametrize("name, before", kernels(), ids=[name for name, _ in kernels()])
def test_both_ctas_run_first(name, before):
    assert 0 <= before.find("cluster_arrive();") < before.find("cluster_wait();")
