"""Edges of the layer operators' calls: what empty rows give."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def oz():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ozaki_ii_fp64_gb300 as oz
    oz.load()
    return oz


@pytest.mark.parametrize("rows", [1, 300])
def test_statistics_of_rows_without_columns(oz, rows):
    # The mean of nothing is 0 / 0; what an earlier tensor left in the memory does not come back.
    x = torch.empty(rows, 0, dtype=BF16, device=DEV)
    for _ in range(3):
        old = [torch.full((rows,), 7.0, device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        del old
        y, mean, rstd = oz.layer_norm(x, stats=True)
        assert y.shape == (rows, 0)
        assert bool(torch.isnan(mean).all()) and bool(torch.isnan(rstd).all())
    assert oz.get_status() == oz.OZEMU_OK
