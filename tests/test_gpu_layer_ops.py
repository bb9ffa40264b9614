"""Layer norm and the fused linear layer on the GPU, forward and backward, against 64-bit references with elementwise
worst-case bounds (layer_reference)."""

import pytest

from layer_reference import linear64, linear_backward64, norm64, norm_backward64, slope64, worst

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


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
    """A rows x cols matrix with leading dimension cols + pad, `offset` elements into its memory; what surrounds it
    is NaN, so that a stray read shows."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ld = cols + pad
    buf = torch.full((rows * ld + offset + 8,), float("nan"), dtype=dtype, device=DEV)
    t = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    t.copy_(torch.randn(rows, cols, generator=gen, device=DEV) * scale)
    return t


def vec(n, dtype, seed, scale=1.0):
    return rnd(1, n, dtype, seed, scale)[0]


# m, k, n: single tokens, few tokens, tile edges on each side, odd and ragged sizes, long sums.
SHAPES = [(1, 1, 1), (1, 8, 8), (1, 4096, 1024), (2, 7, 5), (3, 520, 129), (8, 64, 4104), (13, 1000, 257), (16, 16, 16),
          (17, 64, 33), (31, 2048, 640), (64, 72, 200), (65, 129, 127), (127, 257, 255), (128, 128, 128), (129, 130, 257),
          (255, 512, 384), (300, 65, 1030), (513, 264, 1), (1, 16384, 300), (1500, 33, 520), (2100, 200, 800)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_shapes(oz, shape, dtype):
    m, k, n = shape
    x, w = rnd(m, k, dtype, 1), rnd(n, k, dtype, 2, k ** -0.5)
    b, r = vec(n, dtype, 3), rnd(m, n, dtype, 4)
    y, pre = oz.linear(x, w, b, r, activation="gelu", save_pre=True)
    ref, tol, z, tolz = linear64(x, w, b, r, "gelu")
    assert worst(y, ref, tol) <= 1 and worst(pre, z, tolz) <= 1
    y = oz.linear(x, w)
    ref, tol, _, _ = linear64(x, w)
    assert worst(y, ref, tol) <= 1


# Small outputs of long reductions, which several CTAs share; uneven shares, shares of nothing, edges on both sides.
@pytest.mark.parametrize("m, k, n", [(200, 8192, 136), (513, 4100, 300), (150, 20000, 64), (129, 577, 65), (640, 3000, 256),
                                     (256, 16384, 1024), (100, 9000, 130), (20, 30000, 24), (300, 2000, 2051)])
def test_linear_long_reductions(oz, m, k, n):
    x, w = rnd(m, k, BF16, 101), rnd(n, k, BF16, 102, k ** -0.5)
    b, r = vec(n, BF16, 103), rnd(m, n, BF16, 104)
    y, pre = oz.linear(x, w, b, r, activation="silu", save_pre=True)
    ref, tol, z, tolz = linear64(x, w, b, r, "silu")
    assert worst(y, ref, tol) <= 1 and worst(pre, z, tolz) <= 1
    # The weight gradient's reduction runs over the rows: here k of them.
    dy, x2, w2 = rnd(k, n, BF16, 105, 0.1), rnd(k, m, BF16, 106), rnd(n, m, BF16, 107, 0.1)
    for g, v, e in zip(oz.linear_backward(dy, x2, w2), *linear_backward64(dy, x2, w2)):
        assert worst(g, v, e) <= 1


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [1, 5, 200])
def test_linear_activations(oz, act, m):
    x, w, b = rnd(m, 96, F16, 5, 2.0), rnd(140, 96, F16, 6, 0.2), vec(140, F16, 7, 3.0)
    for res in (None, rnd(m, 140, F16, 8)):
        y, pre = oz.linear(x, w, b, res, activation=act, save_pre=True)
        ref, tol, z, tolz = linear64(x, w, b, res, act)
        assert worst(y, ref, tol) <= 1 and worst(pre, z, tolz) <= 1


@pytest.mark.parametrize("m", [1, 9, 300])
@pytest.mark.parametrize("k, pad, offset", [(64, 8, 0), (64, 3, 0), (64, 8, 1), (61, 3, 0), (61, 0, 5), (136, 0, 8)])
def test_linear_strides_and_alignments(oz, m, k, pad, offset):
    n = 77
    x, w = rnd(m, k, BF16, 9, pad=pad, offset=offset), rnd(n, k, BF16, 10, 0.1, pad=pad, offset=offset)
    r = rnd(m, n, BF16, 11, pad=pad, offset=offset)
    out = rnd(m, n, BF16, 12, pad=5, offset=offset)
    before = out._base.clone()
    y = oz.linear(x, w, None, r, activation="silu", out=out)
    assert y is out
    ref, tol, _, _ = linear64(x, w, None, r, "silu")
    assert worst(y, ref, tol) <= 1
    # What lies round the output is as it was.
    after = out._base.clone()
    torch.as_strided(after, (m, n), (n + 5, 1), offset).fill_(0)
    torch.as_strided(before, (m, n), (n + 5, 1), offset).fill_(0)
    assert torch.equal(after.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("m", [1, 40, 300])
def test_linear_out_may_be_the_residual(oz, m):
    x, w, r = rnd(m, 256, BF16, 13), rnd(192, 256, BF16, 14, 0.06), rnd(m, 192, BF16, 15)
    ref, tol, _, _ = linear64(x, w, None, r.clone(), "relu")
    assert oz.linear(x, w, None, r, activation="relu", out=r) is r
    assert worst(r, ref, tol) <= 1


@pytest.mark.parametrize("m, k, n", [(0, 8, 8), (8, 8, 0), (0, 0, 0), (5, 0, 9), (300, 0, 140)])
def test_linear_empty(oz, m, k, n):
    x, w, b, r = rnd(m, k, BF16, 16), rnd(n, k, BF16, 17), vec(n, BF16, 18), rnd(m, n, BF16, 19)
    y, pre = oz.linear(x, w, b, r, activation="gelu", save_pre=True)
    ref, tol, z, tolz = linear64(x, w, b, r, "gelu")
    assert worst(y, ref, tol) <= 1 and worst(pre, z, tolz) <= 1
    dy = rnd(m, n, BF16, 20)
    got = oz.linear_backward(dy, x, w, pre, activation="gelu")
    want, bounds = linear_backward64(dy, x, w, pre, "gelu")
    for g, v, e in zip(got, want, bounds):
        assert worst(g, v, e) <= 1


@pytest.mark.parametrize("m", [4, 300])
def test_linear_nonfinite_stays_in_its_row_and_column(oz, m):
    x, w, b = rnd(m, 200, BF16, 21), rnd(150, 200, BF16, 22, 0.1), vec(150, BF16, 23)
    clean = oz.linear(x, w, b, activation="relu")
    x2, w2 = x.clone(), w.clone()
    x2[2, 100] = float("nan")
    w2[7, 3] = float("inf")
    y = oz.linear(x2, w2, b, activation="relu")
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[2], keep[:, 7] = False, False
    assert bool(torch.isnan(y[2]).all())
    # An infinite weight gives +inf, relu(-inf) = 0 or NaN by the sign of its factor.
    assert bool((torch.isinf(y[:, 7]) | torch.isnan(y[:, 7]) | (y[:, 7] == 0)).all())
    assert torch.equal(y[keep], clean[keep])


def test_activations_of_large_arguments(oz):
    # z = +-1, +-100, +-1e4, +-1e30: the limits, not inf - inf or 0 * inf.
    z = torch.tensor([[1.0, -1.0, 100.0, -100.0, 1e4, -1e4, 1e30, -1e30]], dtype=BF16, device=DEV).t().contiguous()
    one = torch.ones(1, 1, dtype=BF16, device=DEV)
    for act in ACTS:
        y, pre = oz.linear(z, one, activation=act, save_pre=True)
        ref, tol, _, _ = linear64(z, one, act=act)
        assert torch.equal(pre, z) and worst(y, ref, tol) <= 1
        _, _, db = oz.linear_backward(torch.ones_like(z), z, one, pre, activation=act)
        dx = torch.cat([oz.linear_backward(torch.ones_like(z[i:i + 1]), z[i:i + 1], one, pre[i:i + 1],
                                           activation=act)[0] for i in range(8)])
        s = slope64(z.double().clamp(-1e4, 1e4), act)
        assert float((dx.double() - s).abs().max()) <= 1.2 * 2.0 ** -8 + 2.0 ** -17


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act", ACTS)
def test_slopes_of_infinite_and_nan_arguments(oz, act, dtype):
    # Saved sums that overflowed have the slope's limit; a NaN makes its column's sum NaN and no other.
    big = [float("inf"), float("-inf"), 6e4, -6e4, 40.0, -40.0]
    pre = torch.tensor([big + [float("nan"), 0.5]], dtype=dtype, device=DEV)
    dy, x, w = torch.ones_like(pre), rnd(1, 4, dtype, 240), rnd(8, 4, dtype, 241)
    _, _, db = oz.linear_backward(dy, x, w, pre, activation=act, x_grad=False, w_grad=False)
    assert db[:2].tolist() == [1.0, 1.0 if act == "none" else 0.0]
    s = slope64(pre[0, 2:6].double(), act)
    assert float((db[2:6].double() - s).abs().max()) <= 2.0 ** -8 + 2.0 ** -17
    if act not in ("none", "relu"):
        assert bool(torch.isnan(db[6]))
    assert bool(torch.isfinite(db[7]))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_backward_shapes(oz, shape, dtype):
    m, k, n = shape
    x, w = rnd(m, k, dtype, 31), rnd(n, k, dtype, 32, k ** -0.5)
    dy, pre = rnd(m, n, dtype, 33), rnd(m, n, dtype, 34)
    for act in ("none", "gelu"):
        got = oz.linear_backward(dy, x, w, pre, activation=act)
        want, bounds = linear_backward64(dy, x, w, pre, act)
        for g, v, e in zip(got, want, bounds):
            assert worst(g, v, e) <= 1


@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_activations(oz, act):
    m, k, n = 150, 72, 264
    x, w, dy, pre = rnd(m, k, F16, 35), rnd(n, k, F16, 36, 0.1), rnd(m, n, F16, 37), rnd(m, n, F16, 38, 3.0)
    pre[0, 0], pre[1, 0] = 0.0, -0.0
    got = oz.linear_backward(dy, x, w, pre, activation=act)
    want, bounds = linear_backward64(dy, x, w, pre, act)
    for g, v, e in zip(got, want, bounds):
        assert worst(g, v, e) <= 1


@pytest.mark.parametrize("pad, offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_linear_backward_strides_and_parts(oz, pad, offset):
    m, k, n = 70, 136, 90
    x, w = rnd(m, k, BF16, 39, pad=pad, offset=offset), rnd(n, k, BF16, 40, 0.1, pad=pad, offset=offset)
    dy, pre = rnd(m, n, BF16, 41, pad=pad, offset=offset), rnd(m, n, BF16, 42, pad=pad, offset=offset)
    for act in ("none", "silu"):
        want, bounds = linear_backward64(dy, x, w, pre, act)
        whole = oz.linear_backward(dy, x, w, pre, activation=act)
        for g, v, e in zip(whole, want, bounds):
            assert worst(g, v, e) <= 1
        for part in range(3):  # each gradient alone is the same
            ask = [i == part for i in range(3)]
            got = oz.linear_backward(dy, x, w, pre, activation=act, x_grad=ask[0], w_grad=ask[1], bias_grad=ask[2])
            assert [g is not None for g in got] == ask
            assert torch.equal(got[part], whole[part])


def test_linear_gradient_against_differences(oz):
    # The derivative of sum(dy * linear(x)) along a direction, by differences of the 64-bit formula.
    m, k, n = 33, 40, 50
    x, w, b, dy = rnd(m, k, F16, 43), rnd(n, k, F16, 44, 0.2), vec(n, F16, 45), rnd(m, n, F16, 46)
    _, pre = oz.linear(x, w, b, activation="gelu", save_pre=True)
    got = oz.linear_backward(dy, x, w, pre, activation="gelu")
    _, bounds = linear_backward64(dy, x, w, pre, "gelu")
    from layer_reference import act64
    for which, at in enumerate((x, w, b)):
        v = torch.randn(at.shape, generator=torch.Generator(device=DEV).manual_seed(47), device=DEV,
                        dtype=torch.float64)

        def f(t, which=which):
            p = [x.double(), w.double(), b.double()]
            p[which] = p[which] + t * v
            return float((act64(p[0] @ p[1].t() + p[2], "gelu") * dy.double()).sum())
        h = 1e-5
        slope = (f(h) - f(-h)) / (2 * h)
        # pre is rounded before its slope is taken: |act''| <= 0.8 times u |pre| on every element.
        du = 0.8 * 2.0 ** -11 * pre.double().abs() * dy.double().abs()
        drift = [du @ w.double().abs(), du.t() @ x.double().abs(), du.sum(0)][which]
        room = float(((bounds[which] + drift) * v.abs()).sum()) + 1e-5
        assert abs(slope - float((got[which].double() * v).sum())) <= room


# ---------------------------------------------------------------------------------------------- layer norm

NORM_SHAPES = [(1, 1), (3, 1), (1, 2), (5, 7), (1, 4096), (2, 33), (7, 64), (33, 100), (4, 255), (9, 256), (1, 257),
               (100, 1000), (6, 1024), (5, 1025), (3, 4097), (2, 8192), (2, 12000), (2, 16384), (2, 20001), (1, 40000),
               (1500, 40), (700, 520), (5000, 8)]
TYPES = [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)]


def hidden(rows, cols, dtype, seed, **where):
    t = rnd(rows, cols, dtype, seed, 2.0, **where)
    t.add_(0.5)
    return t


@pytest.mark.parametrize("dtype, wdtype", TYPES, ids=str)
@pytest.mark.parametrize("rows, cols", NORM_SHAPES)
def test_layer_norm_shapes(oz, rows, cols, dtype, wdtype):
    x, w, b = hidden(rows, cols, dtype, 51), vec(cols, wdtype, 52), vec(cols, wdtype, 53)
    got = oz.layer_norm(x, w, b, stats=True)
    want, bounds = norm64(x, w, b)
    for g, v, e in zip(got, want, bounds):
        assert worst(g, v, e) <= 1
    assert torch.equal(oz.layer_norm(x, w, b), got[0])


@pytest.mark.parametrize("dtype, wdtype", TYPES, ids=str)
@pytest.mark.parametrize("rows, cols", NORM_SHAPES)
def test_layer_norm_backward_shapes(oz, rows, cols, dtype, wdtype):
    x, w = hidden(rows, cols, dtype, 54), vec(cols, wdtype, 55)
    dy, dr = rnd(rows, cols, dtype, 56), rnd(rows, cols, dtype, 57)
    (_, mean, rstd), _ = norm64(x, w)
    mean, rstd = mean.float(), rstd.float()
    for extra in (None, dr):
        got = oz.layer_norm_backward(dy, x, mean, rstd, w, dresidual=extra)
        want, bounds = norm_backward64(dy, x, mean, rstd, w, extra)
        for g, v, e in zip(got, want, bounds):
            assert worst(g, v, e) <= 1


# Several rows to a CTA, each taken from its slot twice; in place, as the skip connection's gradient allows.
@pytest.mark.parametrize("rows, cols, dtype, wdtype", [(500, 8200, BF16, BF16), (470, 9001, F16, F32), (330, 16384, BF16, F32),
                                                       (320, 16383, BF16, BF16), (310, 10000, F32, F32)])
def test_layer_norm_backward_of_many_long_rows(oz, rows, cols, dtype, wdtype):
    x, w = hidden(rows, cols, dtype, 250), vec(cols, wdtype, 251)
    dy, dr = rnd(rows, cols, dtype, 252), rnd(rows, cols, dtype, 253)
    (_, mean, rstd), _ = norm64(x, w)
    mean, rstd = mean.float(), rstd.float()
    for extra in (None, dr):
        want, bounds = norm_backward64(dy, x, mean, rstd, w, extra)
        for out in (None, extra):
            got = oz.layer_norm_backward(dy, x, mean, rstd, w, dresidual=extra, out=out)
            for g, v, e in zip(got, want, bounds):
                assert worst(g, v, e) <= 1


@pytest.mark.parametrize("cols, pad, offset", [(64, 8, 0), (64, 3, 0), (61, 0, 5), (520, 8, 1), (1000, 0, 4),
                                               (4099, 5, 0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layer_norm_strides_and_alignments(oz, cols, pad, offset, dtype):
    rows = 11
    where = dict(pad=pad, offset=offset)
    x, dy = hidden(rows, cols, dtype, 58, **where), rnd(rows, cols, dtype, 59, **where)
    dr, w = rnd(rows, cols, dtype, 60, **where), vec(cols + 1, F32, 61)[1:]
    out = rnd(rows, cols, dtype, 62, pad=3, offset=offset)
    before = out._base.clone()
    y, mean, rstd = oz.layer_norm(x, w, stats=True, out=out)
    want, bounds = norm64(x, w)
    for g, v, e in zip((y, mean, rstd), want, bounds):
        assert worst(g, v, e) <= 1
    got = oz.layer_norm_backward(dy, x, mean, rstd, w, dresidual=dr, out=out)
    want, bounds = norm_backward64(dy, x, mean, rstd, w, dr)
    for g, v, e in zip(got, want, bounds):
        assert worst(g, v, e) <= 1
    after = out._base.clone()
    torch.as_strided(after, (rows, cols), (cols + 3, 1), offset).fill_(0)
    torch.as_strided(before, (rows, cols), (cols + 3, 1), offset).fill_(0)
    kind = torch.int32 if dtype == F32 else torch.int16
    assert torch.equal(after.view(kind), before.view(kind))


@pytest.mark.parametrize("cols", [100, 4096, 20001])
def test_layer_norm_without_parameters_and_in_place(oz, cols):
    x = hidden(6, cols, BF16, 63)
    want, bounds = norm64(x)
    orig = x.clone()
    y, mean, rstd = oz.layer_norm(x, stats=True, out=x)
    assert y is x and worst(y, want[0], bounds[0]) <= 1
    b = vec(cols, F32, 64)
    (v, _, _), (e, _, _) = norm64(orig, None, b)
    assert worst(oz.layer_norm(orig, None, b), v, e) <= 1
    dy = rnd(6, cols, BF16, 65)
    want, bounds = norm_backward64(dy, orig, mean, rstd)
    whole = oz.layer_norm_backward(dy, orig, mean, rstd)
    for g, v, e in zip(whole, want, bounds):
        assert worst(g, v, e) <= 1
    only = oz.layer_norm_backward(dy, orig, mean, rstd, weight_grad=False, bias_grad=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], whole[0])
    one = oz.layer_norm_backward(dy, orig, mean, rstd, weight_grad=False)
    assert one[1] is None and torch.equal(one[2], whole[2])
    inplace = oz.layer_norm_backward(dy, orig, mean, rstd, out=dy)
    assert inplace[0] is dy
    for g, v in zip(inplace, whole):
        assert torch.equal(g, v)


@pytest.mark.parametrize("cols", [1, 60, 5000])
def test_layer_norm_empty(oz, cols):
    x, w = hidden(0, cols, BF16, 66), vec(cols, F32, 67)
    y, mean, rstd = oz.layer_norm(x, w, stats=True)
    assert y.shape == (0, cols) and mean.shape == (0,)
    dx, dw, db = oz.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == (0, cols) and not dw.any() and not db.any()
    assert oz.layer_norm(hidden(4, 0, BF16, 68)).shape == (4, 0)


@pytest.mark.parametrize("cols", [96, 3000, 18000])
def test_layer_norm_constant_and_nonfinite_rows(oz, cols):
    x, w, b = hidden(5, cols, F32, 69), vec(cols, F32, 70), vec(cols, F32, 71)
    clean = oz.layer_norm(x, w, b)
    x[1] = 3.0                # no variance: y = b exactly, rstd = eps^-1/2
    x[2, cols // 2] = float("inf")
    x[3, 0] = float("nan")
    y, mean, rstd = oz.layer_norm(x, w, b, stats=True)
    assert torch.equal(y[0], clean[0]) and torch.equal(y[4], clean[4])
    assert float(mean[1]) == 3.0 and abs(float(rstd[1]) * 1e-5 ** 0.5 - 1) < 1e-6
    assert torch.equal(y[1], b)
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())


def test_layer_norm_of_a_large_offset(oz):
    # The variance of values far from 0 is taken round the mean, not as a difference of squares.
    x = rnd(4, 3000, F32, 72) + 1000.0
    want, bounds = norm64(x)
    got = oz.layer_norm(x, stats=True)
    for g, v, e in zip(got, want, bounds):
        assert worst(g, v, e) <= 1


def test_layer_norm_gradient_against_differences(oz):
    rows, cols = 7, 300
    x, w, b, dy = hidden(rows, cols, F32, 73), vec(cols, F32, 74), vec(cols, F32, 75), rnd(rows, cols, F32, 76)
    _, mean, rstd = oz.layer_norm(x, w, b, stats=True)
    got = oz.layer_norm_backward(dy, x, mean, rstd, w)
    for which, at in enumerate((x, w, b)):
        v = torch.randn(at.shape, generator=torch.Generator(device=DEV).manual_seed(77), device=DEV,
                        dtype=torch.float64)

        def f(t, which=which):
            p = [x.double(), w.double(), b.double()]
            p[which] = p[which] + t * v
            d = p[0] - p[0].mean(1, keepdim=True)
            return float((((d / ((d * d).mean(1, keepdim=True) + 1e-5).sqrt()) * p[1] + p[2]) * dy.double()).sum())
        slope = (f(1e-5) - f(-1e-5)) / 2e-5
        # fp32 throughout: 2000 terms of size about 1, each within some 2^-20.
        assert abs(slope - float((got[which].double() * v).sum())) < 2e-3


# ------------------------------------------------------------------------------------------------ both

def test_offsets_beyond_32_bits(oz):
    # 66000 rows, 32776 elements apart: the last row starts past 2^31 elements.
    rows, ld = 66000, 32776
    buf = torch.empty(rows * ld, dtype=BF16, device=DEV)
    x = torch.as_strided(buf, (rows, 64), (ld, 1))
    x.copy_(rnd(rows, 64, BF16, 81))
    w = rnd(24, 64, BF16, 82, 0.1)
    y = torch.as_strided(buf, (rows, 24), (ld, 1), 64)
    oz.linear(x, w, out=y)
    ref, tol, _, _ = linear64(x.contiguous(), w)
    assert worst(y.contiguous(), ref, tol) <= 1
    n = torch.as_strided(buf, (rows, 64), (ld, 1), 128)
    _, mean, rstd = oz.layer_norm(x, out=n, stats=True)
    want, bounds = norm64(x.contiguous())
    assert worst(n.contiguous(), want[0], bounds[0]) <= 1
    dx, dw, db = oz.linear_backward(y, x, w)
    for g, v, e in zip((dx, dw, db), *linear_backward64(y.contiguous(), x.contiguous(), w)):
        assert worst(g, v, e) <= 1
    got = oz.layer_norm_backward(n, x, mean, rstd)
    for g, v, e in zip(got, *norm_backward64(n.contiguous(), x.contiguous(), mean, rstd)):
        assert worst(g, v, e) <= 1


def test_another_stream(oz):
    side = torch.cuda.Stream()
    x, w, b = rnd(300, 512, BF16, 83), rnd(400, 512, BF16, 84, 0.05), vec(400, BF16, 85)
    dy, pre = rnd(300, 400, BF16, 86), rnd(300, 400, BF16, 87)
    here = [oz.linear(x, w, b, activation="gelu"), *oz.linear_backward(dy, x, w, pre, activation="gelu"),
            *oz.layer_norm(x, stats=True)]
    here += oz.layer_norm_backward(x, x, here[-2], here[-1])
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        there = [oz.linear(x, w, b, activation="gelu", stream=side),
                 *oz.linear_backward(dy, x, w, pre, activation="gelu", stream=side),
                 *oz.layer_norm(x, stats=True, stream=side)]
        there += oz.layer_norm_backward(x, x, there[-2], there[-1], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, c in zip(here, there):
        assert torch.equal(a, c)


@pytest.mark.parametrize("m, k, n", [(1, 4096, 512), (40, 2048, 300), (700, 1024, 1024)])
def test_same_bits_every_time(oz, m, k, n):
    x, w, dy = rnd(m, k, BF16, 88), rnd(n, k, BF16, 89, 0.05), rnd(m, n, BF16, 90)
    first = None
    for _ in range(4):
        got = [oz.linear(x, w), *oz.linear_backward(dy, x, w), *oz.layer_norm(x, stats=True)]
        got += oz.layer_norm_backward(x, x, got[-2], got[-1])
        if first is None:
            first = got
        for a, c in zip(first, got):
            assert torch.equal(a, c)


def test_inside_a_cuda_graph(oz):
    # A captured call reads its inputs' memory at each replay.
    x, w, b = rnd(1, 1024, BF16, 91), rnd(512, 1024, BF16, 92, 0.05), vec(512, BF16, 93)
    y, out = torch.empty(1, 1024, dtype=BF16, device=DEV), torch.empty(1, 512, dtype=BF16, device=DEV)

    def step():
        oz.layer_norm(x, out=y)
        oz.linear(y, w, b, activation="silu", out=out)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (94, 95):
        x.copy_(rnd(1, 1024, BF16, seed))
        graph.replay()
        torch.cuda.synchronize()
        ref, tol, _, _ = linear64(y, w, b, None, "silu")
        assert worst(out, ref, tol) <= 1
