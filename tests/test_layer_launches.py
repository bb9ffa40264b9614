"""The layer operators' launches, on the host: a launch that fails ends its call with its error, whatever launch of the
call it is, and an error that another call left pending is not this call's."""

import os
import platform
import subprocess

import pytest

pytest.importorskip("torch")

HERE = os.path.dirname(os.path.abspath(__file__))
WRAPPED = ["cudaLaunchKernelExC", "cudaGetDevice", "cudaFuncSetAttribute", "cudaOccupancyMaxActiveClusters",
           "cudaGetLastError", "cudaGetDriverEntryPointByVersion"]
NO_MEMORY = 2  # cudaErrorMemoryAllocation


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    from ozaki_ii_fp64_gb300 import build
    build.build()
    objects = os.path.join(build.ROOT, "_build", platform.machine())
    exe = str(tmp_path_factory.mktemp("launches") / "host_launches")
    subprocess.run([build.nvcc()] + build.ARCH_FLAGS + ["-std=c++17", "-I" + build.CSRC,
                   os.path.join(HERE, "host_launches.cu"), os.path.join(objects, "linear.o"),
                   os.path.join(objects, "layernorm.o"), "-o", exe]
                   + ["-Xlinker=--wrap=" + name for name in WRAPPED], check=True)

    def run(what, a, b, c=0, odd=0):
        out = subprocess.run([exe, what, str(a), str(b), str(c), str(odd)], check=True, capture_output=True, text=True)
        rows = []
        for line in out.stdout.splitlines():
            status, *grids = line.split()
            rows.append((int(status), [tuple(int(x) for x in g.split(",")) for g in grids]))
        return rows  # without a failure, then with the first launch failing, the second, ...
    return run


@pytest.mark.parametrize("what, a, b, c, odd, count", [
    ("linear", 1000, 4096, 2048, 0, 1), ("linear", 1000, 4096, 2049, 0, 2), ("linear", 3, 4096, 2049, 0, 2),
    ("linear", 5, 9, 0, 0, 1),
    ("linear_backward", 64, 4096, 4096, 0, 3), ("linear_backward", 1000, 1024, 2048, 0, 3),
    ("linear_backward", 1333, 1025, 2051, 0, 4), ("linear_backward", 100000, 264, 264, 0, 4),
    ("linear_backward", 0, 16, 16, 0, 2),
    ("norm", 1, 4096, 0, 0, 1), ("norm", 5000, 1000, 0, 1, 1), ("norm", 10, 70000, 0, 0, 1),
    ("norm_backward", 5000, 1000, 0, 0, 2), ("norm_backward", 100, 20001, 0, 0, 3), ("norm_backward", 0, 1000, 0, 0, 1)])
def test_each_launch_failure_is_the_calls(launches, what, a, b, c, odd, count):
    (status, grids), *failures = launches(what, a, b, c, odd)
    assert status == 0 and len(grids) == count
    assert len(failures) == count
    for i, (status, tried) in enumerate(failures):
        assert status == NO_MEMORY
        assert tried == grids[:i + 1]  # nothing is launched on what was not made


MOST = 2**31 - 2**16  # rows or columns of a norm


@pytest.mark.parametrize("what, a, b, c", [
    ("norm_backward", MOST, 3, 0), ("norm_backward", 2_140_000_000, 1, 0), ("norm_backward", 2_133_400_000, 7, 0),
    ("norm_backward", MOST, 1000, 0), ("norm_backward", 9, MOST, 0), ("norm", MOST, 3, 0), ("norm", MOST, 1000, 0),
    ("norm", 9, MOST, 0), ("linear", 1 << 26, 9, 16), ("linear", 9, 1 << 26, 16), ("linear", 300, 300, 1 << 26),
    ("linear_backward", 1 << 26, 9, 16), ("linear_backward", 9, 1 << 26, 16), ("linear_backward", 300, 300, 1 << 26)])
def test_grids_at_the_size_limits(launches, what, a, b, c):
    # CUDA's limits; a grid that wrapped round is above them.
    (status, grids), *_ = launches(what, a, b, c)
    assert status == 0
    for x, y, z in grids:
        assert 0 < x < 2**31 and 0 < y < 2**16 and 0 < z < 2**16


@pytest.mark.parametrize("rows, cols, odd, first", [
    # Too few rows for the ring's narrow groups: the kernel that keeps a row in registers, not wide groups left idle.
    (300, 256, 0, 75), (912, 64, 0, 228), (3000, 512, 0, 750), (300, 2048, 0, 300), (1000, 63, 1, 250),
    # The ring, one CTA an SM: enough rows for the narrow groups, or rows that fill a share of wide ones.
    (5000, 256, 0, 152), (1000, 1024, 0, 152), (480, 2048, 0, 152), (300, 4096, 0, 152), (300, 2047, 1, 152)])
def test_forward_norm_variant(launches, rows, cols, odd, first):
    (status, grids), *_ = launches("norm", rows, cols, 0, odd)
    assert status == 0 and grids == [(first, 1, 1)]
