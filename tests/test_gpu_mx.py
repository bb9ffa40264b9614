"""Microscaled 4-bit matrices on the GPU: codes, scales and values against a plain restatement, bit for bit, and their
product against 64-bit references with elementwise worst-case bounds (layer_reference)."""

import numpy as np
import pytest

import mx_reference as ref
from layer_reference import TINY, linear64, worst

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


@pytest.fixture(autouse=True)
def clean_status(oz):
    yield
    assert oz.get_status() == oz.OZEMU_OK


def rnd(rows, cols, dtype, seed, scale=1.0, pad=0, offset=0):
    """A matrix with a spread of its own for each row, leading dimension cols + pad, `offset` elements into its memory;
    what surrounds it is NaN, so that a stray read shows."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ld = cols + pad
    buf = torch.full((rows * ld + offset + 8,), float("nan"), dtype=dtype, device=DEV)
    t = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    spread = torch.exp2(6 * torch.rand(rows, 1, generator=gen, device=DEV) - 3)
    t.copy_(torch.randn(rows, cols, generator=gen, device=DEV) * spread * scale)
    return t


def check_quantize(oz, x):
    rows, k = x.shape
    codes, scales = ref.quantize(x.double().cpu().numpy())
    want_codes, want_scales = ref.pack(codes, scales, rows, k)
    q = oz.mx_quantize(x)
    assert q.shape == (rows, k)
    assert np.array_equal(q.codes.cpu().numpy(), want_codes)
    assert np.array_equal(q.scales.cpu().numpy().reshape(want_scales.shape), want_scales)
    v = ref.values(codes, scales)[:, :k]
    for dtype in (x.dtype, F32):
        got = oz.mx_dequantize(q, dtype).double().cpu().numpy()
        assert np.array_equal(got, v, equal_nan=True)
    return q


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows, k", [(1, 1), (1, 32), (3, 31), (2, 33), (1, 4096), (5, 255), (7, 256), (4, 257), (127, 64),
                                     (128, 128), (129, 700), (300, 96), (33, 1000), (260, 513)])
def test_quantize(oz, rows, k, dtype):
    check_quantize(oz, rnd(rows, k, dtype, rows + k))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("pad, offset", [(8, 0), (3, 0), (0, 1), (5, 3), (1, 4), (2, 2)])
def test_quantize_strides(oz, dtype, pad, offset):
    for k in (64, 301):
        check_quantize(oz, rnd(70, k, dtype, 5, pad=pad, offset=offset))


def test_quantize_ties_and_borders(oz):
    # Every middle of two values and the values next to it, of each sign, on scales 2^-20 .. 2^20.
    middles = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.875]
    v = np.array([m * (1 + d) for m in middles for d in (-2.0 ** -7, 0, 2.0 ** -7)] + [0.0, -0.0])
    rows = np.concatenate([np.concatenate([s * v * 2.0 ** e for s in (1, -1)]) for e in (-20, -1, 0, 9)]).reshape(4, -1)
    for first in (4.0, 7.875):  # the largest of each block says the scale
        t = np.zeros((4, 96))
        t[:, :rows.shape[1]] = rows
        t[:, ::32] = first * 2.0 ** np.array([[-20.0], [-1], [0], [9]])
        for dtype in (BF16, F32):
            check_quantize(oz, torch.from_numpy(t).to(DEV).to(dtype))


def test_quantize_extremes(oz):
    # Subnormals, the largest values, zeros, infinities and NaN, each with a block of its own.
    t = torch.zeros(9, 64)
    t[0, :32] = torch.arange(32) * 2.0 ** -133         # subnormal in bfloat16
    t[1, 3], t[1, 40] = 2.0 ** -126, -(2.0 ** -125)
    t[2, :32] = 3.38e38
    t[3, 5] = float("inf")
    t[4, 6] = float("nan")
    t[5, :] = -0.0
    t[6, 7], t[6, 50] = -float("inf"), 1.0
    t[7, :32] = torch.linspace(-1, 1, 32)
    t[8, 0], t[8, 1] = 1.0, 2.0 ** -100
    for dtype in (BF16, F32):
        q = check_quantize(oz, t.to(dtype).to(DEV))
        assert torch.isnan(oz.mx_dequantize(q)[3:5, :32]).all()
    h = torch.zeros(4, 32)
    h[0, :] = torch.arange(32) * 2.0 ** -24            # subnormal in float16
    h[1, :] = 65504.0
    h[2, 1] = float("nan")
    h[3, 9] = -float("inf")
    check_quantize(oz, h.to(F16).to(DEV))


def test_quantize_of_held_values_keeps_them(oz):
    x = rnd(50, 200, BF16, 8)
    y = oz.mx_dequantize(oz.mx_quantize(x))
    assert torch.equal(oz.mx_dequantize(oz.mx_quantize(y)), y)


def test_quantize_into_memory_that_is_there(oz):
    x = rnd(40, 100, BF16, 9)
    q = oz.mx_quantize(rnd(40, 100, BF16, 10))
    data = q.data
    assert oz.mx_quantize(x, out=q) is q and q.data is data
    fresh = oz.mx_quantize(x)
    assert torch.equal(q.codes, fresh.codes) and torch.equal(q.scales, fresh.scales)
    empty = oz.mx_quantize(x, out=oz.MXMatrix.empty(40, 100))
    assert torch.equal(empty.codes, fresh.codes) and torch.equal(empty.scales, fresh.scales)
    y = rnd(40, 100, F32, 11, pad=3)
    before = y._base.clone()
    assert oz.mx_dequantize(q, out=y) is y
    assert torch.equal(y, oz.mx_dequantize(q, F32))
    after = y._base.clone()
    for t in (before, after):  # what lies round the output is as it was
        torch.as_strided(t, (40, 100), (103, 1), 0).fill_(0)
    assert torch.equal(after.view(torch.int32), before.view(torch.int32))


def product(oz, m, k, n, dtype, act="none", bias=True, residual=False, seed=20):
    x, w = rnd(m, k, dtype, seed), rnd(n, k, dtype, seed + 1, k ** -0.5)
    b = rnd(1, n, dtype, seed + 2)[0] if bias else None
    r = rnd(m, n, dtype, seed + 3) if residual else None
    xq, wq = oz.mx_quantize(x), oz.mx_quantize(w)
    y = oz.mx_linear(xq, wq, b, r, activation=act, dtype=dtype)
    want, tol, _, _ = linear64(oz.mx_dequantize(xq, dtype), oz.mx_dequantize(wq, dtype), b, r, act)
    assert worst(y, want, tol) <= 1
    return y


# Single tokens, few tokens, tile edges on each side, odd and ragged sizes, long sums, both tile widths.
SHAPES = [(1, 1, 1), (1, 32, 8), (1, 4096, 1024), (2, 7, 5), (3, 520, 129), (8, 64, 4104), (13, 1000, 257), (16, 16, 16),
          (17, 64, 33), (31, 2048, 640), (64, 72, 200), (65, 129, 127), (127, 257, 255), (128, 128, 128), (129, 130, 257),
          (255, 512, 384), (300, 65, 1030), (513, 264, 1), (1, 16384, 300), (1500, 33, 520), (2100, 200, 800),
          (1300, 1000, 2500), (2000, 700, 6000), (5000, 260, 4100)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_product_shapes(oz, shape, dtype):
    m, k, n = shape
    product(oz, m, k, n, dtype, "gelu", residual=True)
    product(oz, m, k, n, dtype, bias=False)


# Reductions that a cluster shares, unevenly, for every number of rows that it takes, and few rows of short ones.
@pytest.mark.parametrize("m, k, n", [(16, 8200, 130), (30, 2048, 200), (30, 1700, 264), (32, 9000, 1000), (50, 4100, 77),
                                     (64, 4352, 640), (60, 5000, 129), (100, 8200, 130), (128, 9001, 256), (90, 7000, 300),
                                     (200, 8192, 136), (300, 16384, 300), (150, 20000, 64), (1000, 8192, 512)])
def test_product_long_reductions(oz, m, k, n):
    product(oz, m, k, n, BF16, "silu", residual=True)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m", [1, 40, 700])
def test_product_activations(oz, act, m):
    product(oz, m, 200, 2300, F16, act)
    product(oz, m, 200, 2300, BF16, act, bias=False, residual=True)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m, k, n, pad", [(1, 200, 300, 0), (40, 300, 2048, 8), (500, 256, 2049, 0), (700, 300, 2304, 0),
                                          (700, 300, 2304, 5)])
def test_product_times_a_matrix(oz, m, k, n, pad, dtype):
    # With the other half's product as the factor: a gated layer.
    x, gate, up = rnd(m, k, dtype, 60, 0.5), rnd(n, k, dtype, 61, k ** -0.5), rnd(n, k, dtype, 62, k ** -0.5)
    b = rnd(1, n, dtype, 63)[0]
    xq, gq, uq = oz.mx_quantize(x), oz.mx_quantize(gate), oz.mx_quantize(up)
    u = oz.mx_linear(xq, uq, dtype=dtype, out=rnd(m, n, dtype, 64, pad=pad))
    h = oz.mx_linear(xq, gq, b, activation="silu", times=u)
    a, tol, _, _ = linear64(oz.mx_dequantize(xq, dtype), oz.mx_dequantize(gq, dtype), b, None, "silu")
    # tol is u |a| + (1 + u) e of the rounded a; the product has e |u|, an fp32 rounding and its own to the type.
    want = a * u.double()
    bound = tol * u.double().abs() + 2.0 ** -23 * want.abs() + TINY[dtype]
    assert worst(h, want, bound) <= 1
    assert oz.mx_linear(xq, gq, b, activation="silu", times=u, out=u) is u
    assert torch.equal(u, h)


def test_product_takes_every_scale_of_its_own_block(oz):
    # One element of a block is 1 and its scale a power of two that only this row and block have: an output says which
    # scales met.
    for m, n in ((16, 256), (300, 6000)):
        k = 1024
        x, w = torch.zeros(m, k, device=DEV), torch.zeros(n, k, device=DEV)
        i, j = torch.arange(m, device=DEV), torch.arange(n, device=DEV)
        blocks = torch.arange(k // 32, device=DEV)
        x[:, blocks * 32 + 5] = torch.exp2(((i[:, None] * 7 + blocks * 3) % 11 - 5).float())
        w[:, blocks * 32 + 5] = torch.exp2(((j[:, None] * 5 + blocks * 2) % 13 - 6).float())
        y = oz.mx_linear(oz.mx_quantize(x), oz.mx_quantize(w), dtype=F16)
        want = x.double() @ w.double().t()
        assert worst(y, want, 2.0 ** -11 * want.abs()) <= 1  # sums of 32 powers of two: exact in fp32


def test_product_of_nan_blocks(oz):
    for m in (4, 400):
        x, w = rnd(m, 300, BF16, 30), rnd(2500, 300, BF16, 31)
        x[1, 299] = float("nan")
        w[2100, 0] = float("inf")
        y = oz.mx_linear(oz.mx_quantize(x), oz.mx_quantize(w))
        nan = torch.isnan(y)
        want = torch.zeros_like(nan)
        want[1, :] = True
        want[:, 2100] = True
        assert torch.equal(nan, want)


def test_product_of_nothing(oz):
    empty = oz.mx_quantize(torch.empty(3, 0, dtype=BF16, device=DEV))
    weights = oz.mx_quantize(torch.empty(5, 0, dtype=BF16, device=DEV))
    b = rnd(1, 5, BF16, 1)[0]
    y = oz.mx_linear(empty, weights, b, activation="relu")
    assert torch.equal(y, b.clamp(min=0).expand(3, 5))
    assert oz.mx_linear(oz.mx_quantize(rnd(1, 64, BF16, 2)[:0]), oz.mx_quantize(rnd(4, 64, BF16, 3))).shape == (0, 4)
    t = rnd(3, 5, BF16, 4)
    assert torch.equal(oz.mx_linear(empty, weights, b, times=t), (b.float() * t.float()).bfloat16())
    assert torch.equal(oz.mx_linear(empty, weights, residual=t), t)
    assert oz.mx_dequantize(empty).shape == (3, 0)


def test_product_into_its_residual_and_strides(oz):
    for m in (3, 500):
        x, w = rnd(m, 100, BF16, 40), rnd(2100, 100, BF16, 41, 0.1)
        xq, wq = oz.mx_quantize(x), oz.mx_quantize(w)
        r = rnd(m, 2100, BF16, 42, pad=5, offset=1)
        want = oz.mx_linear(xq, wq, residual=r)
        before = r._base.clone()
        assert oz.mx_linear(xq, wq, residual=r, out=r) is r
        assert torch.equal(r, want)
        after = r._base.clone()
        for t in (before, after):
            torch.as_strided(t, (m, 2100), (2105, 1), 1).fill_(0)
        assert torch.equal(after.view(torch.int16), before.view(torch.int16))


def test_products_repeat_bit_for_bit_on_streams_and_in_graphs(oz):
    x, w = rnd(600, 1000, BF16, 50), rnd(3000, 1000, BF16, 51, 0.03)
    one = rnd(1, 1000, BF16, 52)
    wq = oz.mx_quantize(w)
    want, want1 = oz.mx_linear(oz.mx_quantize(x), wq), oz.mx_linear(oz.mx_quantize(one), wq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = oz.mx_linear(oz.mx_quantize(x, stream=side), wq, stream=side)
    y1 = oz.mx_linear(oz.mx_quantize(one), wq)  # at the same time
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want) and torch.equal(y1, want1)
    graph = torch.cuda.CUDAGraph()
    held = x.clone()
    with torch.cuda.graph(graph):
        g = oz.mx_linear(oz.mx_quantize(held), wq)
        g1 = oz.mx_linear(oz.mx_quantize(one), wq)
    for _ in range(2):
        graph.replay()
    assert torch.equal(g, want) and torch.equal(g1, want1)
    held.neg_()
    graph.replay()
    assert torch.equal(g, oz.mx_linear(oz.mx_quantize(-x), wq))
