"""Edges of the layer operators' calls: empty rows, outputs in the place of inputs."""

import warnings

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


@pytest.mark.parametrize("rows, cols", [(5, 7), (700, 520), (3000, 1001), (1600, 4096), (500, 8200), (320, 16383), (100, 20001),
                                        (60, 24000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_gradient_in_the_place_of_x(oz, rows, cols, dtype):
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, dy, dr = (torch.randn(rows, cols, generator=gen, device=DEV).to(dtype) for _ in range(3))
    w = torch.randn(cols, generator=gen, device=DEV)
    _, mean, rstd = oz.layer_norm(x, w, stats=True)
    for extra in (None, dr):
        want = oz.layer_norm_backward(dy, x, mean, rstd, w, dresidual=extra)
        place = x.clone()
        got = oz.layer_norm_backward(dy, place, mean, rstd, w, dresidual=extra, out=place)
        assert got[0] is place
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert oz.get_status() == oz.OZEMU_OK


def test_overlapping_output_is_refused(oz):
    x, w = torch.randn(64, 64, device=DEV).to(BF16), torch.randn(64, 64, device=DEV).to(BF16)
    before = x.clone()
    for call in (lambda: oz.linear(x, w, out=x), lambda: oz.linear(x, w, out=w), lambda: oz.layer_norm(x[1:], out=x[:-1])):
        with pytest.raises(ValueError, match="overlaps"):
            call()
    assert torch.equal(x, before)
    wide = torch.randn(64, 192, device=DEV).to(BF16)  # columns of one matrix share nothing
    y = oz.linear(wide[:, :64], w, residual=wide[:, 64:128], out=wide[:, 128:])
    assert torch.equal(y, oz.linear(wide[:, :64].clone(), w, residual=wide[:, 64:128].clone()))


def test_inputs_that_require_gradients_are_answered_with_a_warning(oz):
    x, w = torch.randn(4, 64, device=DEV).to(BF16), torch.nn.Parameter(torch.randn(32, 64, device=DEV).to(BF16))
    gain = torch.nn.Parameter(torch.ones(64, device=DEV))
    dy, mean, rstd = torch.ones(4, 32, dtype=BF16, device=DEV), torch.zeros(4, device=DEV), torch.ones(4, device=DEV)
    calls = {"linear": lambda: oz.linear(x, w), "linear_backward": lambda: oz.linear_backward(dy, x, w)[0],
             "layer_norm": lambda: oz.layer_norm(x, gain),
             "layer_norm_backward": lambda: oz.layer_norm_backward(x, x, mean, rstd, gain)[0]}
    for name, call in calls.items():
        with pytest.warns(UserWarning, match="^%s: an input requires a gradient" % name):
            loud = call()
        assert not loud.requires_grad
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with pytest.raises(UserWarning):
                call()
            with torch.no_grad():
                assert torch.equal(call(), loud)
    with warnings.catch_warnings():  # and none where nothing requires one
        warnings.simplefilter("error")
        oz.linear(x, w.detach())
        oz.layer_norm(x, gain.detach())
    assert oz.get_status() == oz.OZEMU_OK
