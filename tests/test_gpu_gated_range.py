"""Gradients of the gated layer over float16's whole range: dz = [dh u act'(g)  dh act(g)], a product of three, leaves it
where dh, x, w and the gradients themselves do not."""

import math

import pytest

from layer_reference import act64, slope64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F16 = torch.float16
U = 2.0 ** -11     # a rounding to float16, relative
TINY = 2.0 ** -25  # and the largest of a subnormal result


@pytest.fixture(scope="module")
def oz():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ozaki_ii_fp64_gb300 as oz
    oz.load()
    return oz


@pytest.fixture(autouse=True)
def clean_status(oz):
    yield
    assert oz.get_status() == oz.OZEMU_OK


def rnd(rows, cols, seed, scale=1.0, pad=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(rows, cols + pad, generator=gen, device=DEV) * scale).to(F16)[:, :cols]


def gradients64(dh, x, w, pre, act):
    n = dh.shape[1]
    d, g, u = dh.double(), pre.double()[:, :n], pre.double()[:, n:]
    dz = torch.cat((d * u * slope64(g, act), d * act64(g, act)), 1)
    return dz @ w.double(), dz.t() @ x.double(), dz.sum(0)


def near(got, want, roundings=2):
    """Two roundings, of dz and of the result: each adds at most U of what it rounds, in 2-norm (a sum of many terms does
    not amplify a relative error of independent roundings); a subnormal result TINY an element.  What fp32 adds is within
    the half that a rounding's error stays below its bound on average."""
    assert bool(torch.isfinite(got).all())
    error = float((got.double() - want).norm())
    return error <= roundings * U * float(want.norm()) + TINY * math.sqrt(want.numel())


# Whole rows, odd ones, few rows, reductions that CTA pairs share (of dx: 256 rows; of dw: 8192), one token.
SHAPES = [(1024, 256, 256), (300, 65, 77), (40, 512, 1024), (256, 512, 4096), (8192, 520, 256), (1333, 2051, 1025), (1, 64, 40),
          (700, 8, 3)]


@pytest.mark.parametrize("scale", [1.0, 1e-5, 1e-6])
@pytest.mark.parametrize("m, k, n", SHAPES)
def test_small_gradients(oz, m, k, n, scale):
    dh, x, w, pre = rnd(m, n, 1, scale), rnd(m, k, 2), rnd(2 * n, k, 3), rnd(m, 2 * n, 4)
    for got, want in zip(oz.gated_linear_backward(dh, x, w, pre), gradients64(dh, x, w, pre, "silu")):
        assert near(got, want)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m, n, pad", [(100, 64, 0), (600, 256, 8), (600, 131, 1)])
def test_activations(oz, act, m, n, pad):
    dh, x, w, pre = rnd(m, n, 5, 3e-6, pad), rnd(m, 96, 6, pad=pad), rnd(2 * n, 96, 7, pad=pad), rnd(m, 2 * n, 8, 0.3, pad)
    for got, want in zip(oz.gated_linear_backward(dh, x, w, pre, activation=act), gradients64(dh, x, w, pre, act)):
        assert near(got, want)


@pytest.mark.parametrize("m, n", [(100, 64), (600, 256), (600, 131)])
def test_products_beyond_the_largest_float16(oz, m, n):
    # dz of up to 4e5; dx, dw and db within the type.
    dh, x, w, pre = rnd(m, n, 9, 300.0), rnd(m, 96, 10, 1e-3), rnd(2 * n, 96, 11, 1e-3), rnd(m, 2 * n, 12, 300.0)
    want = gradients64(dh, x, w, pre, "silu")
    dz = dh.double() * pre.double()[:, n:]
    assert float(dz.abs().max()) > 2e5 and max(float(v.abs().max()) for v in want[:2]) < 6e4
    for got, v in zip(oz.gated_linear_backward(dh, x, w, pre, bias_grad=False)[:2], want):
        assert near(got, v)


def test_tokens_of_every_size(oz):
    # Rows of dh from 1 down to 2^-20 keep their relative error, each its own.
    m, n, k = 512, 256, 256
    dh = (rnd(m, n, 13).float() * torch.exp2(-20 * torch.arange(m, device=DEV) / (m - 1)).unsqueeze(1)).to(F16)
    x, w, pre = rnd(m, k, 14), rnd(2 * n, k, 15, 8.0), rnd(m, 2 * n, 16)
    dx, dw, db = oz.gated_linear_backward(dh, x, w, pre)
    want = gradients64(dh, x, w, pre, "silu")
    for i in range(m):
        assert near(dx[i], want[0][i])
    assert near(dw, want[1]) and near(db, want[2])


def test_infinities_keep_to_their_rows(oz):
    for m in (60, 300):
        x, w, dh, pre = rnd(m, 64, 30), rnd(80, 64, 31), rnd(m, 40, 32, 1e-6), rnd(m, 80, 33)
        want = gradients64(dh, x, w, pre, "silu")
        pre[7, 43] = float("inf")  # u of column 3
        dh[11, 5] = float("nan")
        dx, dw, db = oz.gated_linear_backward(dh, x, w, pre)
        good = torch.ones(m, dtype=torch.bool, device=DEV)
        good[7] = good[11] = False
        assert torch.equal(torch.isfinite(dx).all(1), good) and near(dx[good], want[0][good])
        good = torch.ones(80, dtype=torch.bool, device=DEV)
        good[3] = good[5] = good[45] = False
        assert torch.equal(torch.isfinite(dw).all(1), good) and torch.equal(torch.isfinite(db), good)


def test_of_zeros(oz):
    for m in (3, 300):
        x, w, pre = rnd(m, 64, 40), rnd(80, 64, 41), rnd(m, 80, 42)
        for g in oz.gated_linear_backward(torch.zeros(m, 40, dtype=F16, device=DEV), x, w, pre):
            assert not g.any()


def test_repeats_on_streams_and_in_graphs(oz):
    m, n, k = 600, 256, 128
    x, w, pre, dh = rnd(m, k, 50), rnd(2 * n, k, 51), rnd(m, 2 * n, 52), rnd(m, n, 53, 1e-6)
    other = (dh.float() * 5e4).to(F16)
    want, want_other = oz.gated_linear_backward(dh, x, w, pre), oz.gated_linear_backward(other, x, w, pre)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there, here = oz.gated_linear_backward(other, x, w, pre, stream=side), oz.gated_linear_backward(dh, x, w, pre)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(g, v) for g, v in zip(there, want_other)) and all(torch.equal(g, v) for g, v in zip(here, want))
    held = dh.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = oz.gated_linear_backward(held, x, w, pre)
    for value, expected in ((dh, want), (other, want_other), (dh, want)):  # each replay finds its own scale
        held.copy_(value)
        graph.replay()
        assert all(torch.equal(g, v) for g, v in zip(got, expected))
