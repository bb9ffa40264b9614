"""A group of threads that waits for a slot leaves together when some of its threads give up.

The probe's waits run out after 2 ms on a slot that nothing fills; no copy is in flight."""

import ctypes
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
LIMIT_NS = 2_000_000
TIMEOUT_FLAG = 2  # kFlagTimeout in common.cuh


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from ozaki_ii_fp64_gb300 import build
    so = str(tmp_path_factory.mktemp("probe") / "slot_wait_probe.so")
    subprocess.run([build.nvcc()] + build.ARCH_FLAGS + ["-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
                   "-I" + build.CSRC, os.path.join(HERE, "slot_wait_probe.cu"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.probe.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_ulonglong, ctypes.POINTER(ctypes.c_int)]

    def run(threads, mask, value):
        out = (ctypes.c_int * 7)()
        assert lib.probe(threads, mask, value, LIMIT_NS, out) == 0
        return list(out)
    return run


@pytest.mark.parametrize("threads", [32, 128, 512])
@pytest.mark.parametrize("which", ["odd", "last", "all"])
def test_a_group_gives_up_together(probe, threads, which):
    mask, value = {"odd": (1, 1), "last": (threads - 1, threads - 1), "all": (0, 0)}[which]
    out = probe(threads, mask, value)
    assert out[:2] == [0, threads]       # the group whose slot is filled goes on, whole
    assert out[2:4] == [threads, 0]      # the other leaves, whole
    assert out[4] == threads and out[6] & TIMEOUT_FLAG


def test_no_group_gives_up_without_a_cause(probe):
    assert probe(128, 0, 1) == [0, 128, 0, 128, 128, 128, 0]  # nobody waits for the empty slot


@pytest.mark.parametrize("rows, cols", [(6000, 256), (3000, 1001), (2000, 4096), (1000, 12000)])
def test_norms_end_under_a_timeout_of_another_call(rows, cols):
    # The flag is the device's: waits that poll while it stands may give up.  The calls end, the status tells, and
    # the next calls are right.
    import ozaki_ii_fp64_gb300 as oz
    stream = torch.cuda.current_stream().cuda_stream
    x = torch.randn(rows, cols, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda").bfloat16()
    y, mean, rstd = oz.layer_norm(x, stats=True)
    grads = oz.layer_norm_backward(x, x, mean, rstd)
    assert oz.get_status() == oz.OZEMU_OK
    assert oz.ozemu_probe_wait_timeout(LIMIT_NS, stream) == oz.OZEMU_OK
    for _ in range(3):
        oz.layer_norm(x, stats=True)
        oz.layer_norm_backward(x, x, mean, rstd)
    assert oz.get_status() == oz.OZEMU_ERR_TIMEOUT
    again = [*oz.layer_norm(x, stats=True), *oz.layer_norm_backward(x, x, mean, rstd)]
    assert oz.get_status() == oz.OZEMU_OK
    for a, b in zip((y, mean, rstd, *grads), again):
        assert torch.equal(a, b)
