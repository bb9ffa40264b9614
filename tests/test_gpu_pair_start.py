"""Pair kernels that start while other streams' kernels fill the GPU, over and over: the product's operands are split on one
stream beside the GEMMs of the chunks before on another, and the layers' products beside copies."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def oz():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ozaki_ii_fp64_gb300 as oz
    oz.load()
    return oz


@pytest.mark.parametrize("m, n, k, r, times", [(4096, 4096, 65536, 17, 20), (4096, 2048, 16384, 17, 60)])
def test_products_of_chunks_beside_their_splits(oz, m, n, k, r, times):
    gen = torch.Generator(device=DEV).manual_seed(1)
    A = torch.randn(m, k, generator=gen, device=DEV, dtype=torch.float64)
    B = torch.randn(k, n, generator=gen, device=DEV, dtype=torch.float64)
    C, first = torch.empty(m, n, device=DEV, dtype=torch.float64), None
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(times):
        assert oz.ozemu_dgemm_mixed(m, n, k, A.data_ptr(), k, B.data_ptr(), n, C.data_ptr(), n, r, stream) == oz.OZEMU_OK
        torch.cuda.synchronize()
        first = C.clone() if first is None else first
        assert torch.equal(C.view(torch.int64), first.view(torch.int64))
    assert oz.get_status() == oz.OZEMU_OK


def test_layers_beside_copies(oz):
    gen = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(1000, 1024, generator=gen, device=DEV).bfloat16()
    w = (torch.randn(4096, 1024, generator=gen, device=DEV) / 32).bfloat16()
    xq, wq = oz.mx_quantize(x), oz.mx_quantize(w)
    want = oz.linear(x, w), oz.gated_linear(x, w), oz.mx_linear(xq, wq)
    busy = torch.ones(1 << 26, device=DEV)
    torch.cuda.synchronize()
    for _ in range(50):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(4):
                busy.mul_(1.0)
        got = oz.linear(x, w), oz.gated_linear(x, w), oz.mx_linear(xq, wq)
        torch.cuda.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got, want))
    assert oz.get_status() == oz.OZEMU_OK
