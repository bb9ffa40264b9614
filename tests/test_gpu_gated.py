"""The gated linear layer on the GPU, forward and backward, against 64-bit references with elementwise worst-case bounds
(layer_reference)."""

import pytest

from layer_reference import ACT, EPS, TINY, U, act64, slope64, worst

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F16 = torch.bfloat16, torch.float16
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
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ld = cols + pad
    buf = torch.full((rows * ld + offset + 8,), float("nan"), dtype=dtype, device=DEV)
    t = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    t.copy_(torch.randn(rows, cols, generator=gen, device=DEV) * scale)
    return t


def gated64(x, w, b, act):
    """(h, its bound, z, its bound): z's fp32 sums as linear64 bounds them, the activation's error ACT |g|, slopes up to
    1.2, the product's EPS, and the rounding."""
    u, tiny = U[x.dtype], TINY[x.dtype]
    xd, wd = x.double(), w.double()
    z, mag = xd @ wd.t(), xd.abs() @ wd.abs().t()
    if b is not None:
        z, mag = z + b.double(), mag + b.double().abs()
    ez = (x.shape[1] + 2) * EPS * mag
    (g, up), (eg, eu) = z.chunk(2, 1), ez.chunk(2, 1)
    a, ea = act64(g, act), 1.2 * eg + ACT * g.abs()
    h = a * up
    eh = ea * up.abs() + (a.abs() + ea) * eu + EPS * h.abs()
    return h, u * h.abs() + (1 + u) * eh + tiny, z, u * z.abs() + (1 + u) * ez + tiny


def gated_backward64(dh, x, w, pre, act):
    """((dx, dw, db), their bounds): dz is rounded to the type for the products, not for db."""
    u, tiny = U[x.dtype], TINY[x.dtype]
    m, n = dh.shape
    xd, wd, d = x.double(), w.double(), dh.double()
    g, up = pre.double()[:, :n], pre.double()[:, n:]
    dz = torch.cat((d * up * slope64(g, act), d * act64(g, act)), 1)
    edz = torch.cat((2 * ACT * (d * up).abs() + 2 * EPS * dz[:, :n].abs(), ACT * (d * g).abs() + EPS * dz[:, n:].abs()), 1)
    erd = edz + u * (dz.abs() + edz) + tiny
    zmag = dz.abs() + erd
    dx, edx = dz @ wd, erd @ wd.abs() + (2 * n + 2) * EPS * (zmag @ wd.abs())
    dw, edw = dz.t() @ xd, erd.t() @ xd.abs() + (m + 2) * EPS * (zmag.t() @ xd.abs())
    db, edb = dz.sum(0), edz.sum(0) + (m + 2) * EPS * zmag.sum(0)

    def done(v, e):
        return u * v.abs() + (1 + u) * e + tiny
    return (dx, dw, db), (done(dx, edx), done(dw, edw), done(db, edb))


SHAPES = [(1, 1, 1), (1, 8, 8), (1, 4096, 1024), (2, 7, 5), (3, 520, 129), (8, 64, 4104), (13, 1000, 257), (16, 16, 16),
          (17, 64, 33), (31, 2048, 640), (64, 72, 200), (65, 129, 127), (127, 257, 255), (128, 128, 128), (129, 130, 257),
          (255, 512, 384), (300, 65, 1030), (513, 264, 1), (1, 16384, 300), (1500, 33, 520), (2100, 200, 800),
          (700, 100, 2049), (400, 16384, 200), (640, 9000, 130)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(oz, shape, dtype):
    m, k, n = shape
    x, w, b = rnd(m, k, dtype, 1), rnd(2 * n, k, dtype, 2, k ** -0.5), rnd(1, 2 * n, dtype, 3)[0]
    h, pre = oz.gated_linear(x, w, b, save_pre=True)
    want, tol, z, tolz = gated64(x, w, b, "silu")
    assert worst(h, want, tol) <= 1 and worst(pre, z, tolz) <= 1
    h = oz.gated_linear(x, w)
    want, tol, _, _ = gated64(x, w, None, "silu")
    assert worst(h, want, tol) <= 1
    dh = rnd(m, n, dtype, 4)
    pre = rnd(m, 2 * n, dtype, 5)
    for got, v, e in zip(oz.gated_linear_backward(dh, x, w, pre), *gated_backward64(dh, x, w, pre, "silu")):
        assert worst(got, v, e) <= 1


# Long reductions of few tiles, which two or four CTA pairs share; more than the kernel for few rows takes, and that kernel's.
@pytest.mark.parametrize("m, k, n", [(256, 8192, 2600), (250, 6000, 2601), (130, 20000, 3000), (256, 3000, 2560), (100, 1500, 700),
                                     (128, 9000, 136), (64, 9000, 136), (300, 16384, 1700), (512, 8192, 1300)])
def test_long_reductions(oz, m, k, n):
    x, w, b = rnd(m, k, BF16, 61), rnd(2 * n, k, BF16, 62, k ** -0.5), rnd(1, 2 * n, BF16, 63)[0]
    h, pre = oz.gated_linear(x, w, b, activation="gelu", save_pre=True)
    want, tol, z, tolz = gated64(x, w, b, "gelu")
    assert worst(h, want, tol) <= 1 and worst(pre, z, tolz) <= 1
    assert torch.equal(oz.gated_linear(x, w, b, activation="gelu"), h)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [1, 5, 200, 700])
def test_activations(oz, act, m):
    x, w, b = rnd(m, 96, F16, 5, 2.0), rnd(280, 96, F16, 6, 0.2), rnd(1, 280, F16, 7, 3.0)[0]
    h, pre = oz.gated_linear(x, w, b, activation=act, save_pre=True)
    want, tol, z, tolz = gated64(x, w, b, act)
    assert worst(h, want, tol) <= 1 and worst(pre, z, tolz) <= 1
    dh = rnd(m, 140, F16, 8)
    for got, v, e in zip(oz.gated_linear_backward(dh, x, w, pre, activation=act),
                         *gated_backward64(dh, x, w, pre, act)):
        assert worst(got, v, e) <= 1


@pytest.mark.parametrize("m", [1, 9, 300])
@pytest.mark.parametrize("k, n, pad, offset", [(64, 80, 8, 0), (64, 77, 3, 0), (64, 80, 8, 1), (61, 76, 3, 0), (61, 77, 0, 5),
                                               (136, 72, 0, 8), (64, 76, 8, 0)])
def test_strides_and_alignments(oz, m, k, n, pad, offset):
    x, w = rnd(m, k, BF16, 9, pad=pad, offset=offset), rnd(2 * n, k, BF16, 10, 0.1, pad=pad, offset=offset)
    b = rnd(1, 2 * n, BF16, 13, offset=offset)[0]
    out = rnd(m, n, BF16, 12, pad=5, offset=offset)
    before = out._base.clone()
    assert oz.gated_linear(x, w, b, out=out) is out
    want, tol, _, _ = gated64(x, w, b, "silu")
    assert worst(out, want, tol) <= 1
    after = out._base.clone()  # what lies round the output is as it was
    for t in (before, after):
        torch.as_strided(t, (m, n), (n + 5, 1), offset).fill_(0)
    assert torch.equal(after.view(torch.int16), before.view(torch.int16))
    dh, pre = rnd(m, n, BF16, 14, pad=pad, offset=offset), rnd(m, 2 * n, BF16, 15, pad=pad, offset=offset)
    for got, v, e in zip(oz.gated_linear_backward(dh, x, w, pre), *gated_backward64(dh, x, w, pre, "silu")):
        assert worst(got, v, e) <= 1


def test_which_gradients(oz):
    x, w, pre, dh = rnd(300, 64, BF16, 20), rnd(80, 64, BF16, 21), rnd(300, 80, BF16, 22), rnd(300, 40, BF16, 23)
    dx, dw, db = oz.gated_linear_backward(dh, x, w, pre)
    for i in range(8):
        got = oz.gated_linear_backward(dh, x, w, pre, x_grad=bool(i & 1), w_grad=bool(i & 2), bias_grad=bool(i & 4))
        for g, want, asked in zip(got, (dx, dw, db), (i & 1, i & 2, i & 4)):
            assert (g is None) if not asked else torch.equal(g, want)


def test_of_nothing(oz):
    x, w, b = rnd(3, 0, BF16, 1), rnd(8, 0, BF16, 2), rnd(1, 8, BF16, 3)[0]
    h, pre = oz.gated_linear(x, w, b, activation="relu", save_pre=True)
    assert torch.equal(pre, b.expand(3, 8))
    assert torch.equal(h, (b[:4].float().clamp(min=0) * b[4:].float()).bfloat16().expand(3, 4))
    assert oz.gated_linear(rnd(1, 16, BF16, 4)[:0], rnd(8, 16, BF16, 5)).shape == (0, 4)
    dx, dw, db = oz.gated_linear_backward(rnd(1, 4, BF16, 6)[:0], rnd(1, 16, BF16, 7)[:0], rnd(8, 16, BF16, 8),
                                          rnd(1, 8, BF16, 9)[:0])
    x, w = rnd(3, 16, BF16, 10), rnd(1, 16, BF16, 11)[:0]
    empty = torch.empty(3, 0, dtype=BF16, device=DEV)
    assert oz.gated_linear(x, w).shape == (3, 0)
    gx, gw, gb = oz.gated_linear_backward(empty, x, w, empty)
    assert gx.shape == (3, 16) and not gx.any() and gw.shape == (0, 16) and gb.shape == (0,)
    assert dx.shape == (0, 16) and not dw.any() and not db.any() and dw.shape == (8, 16) and db.shape == (8,)


def test_infinities_and_nan(oz):
    # g infinite: silu and its slope have limits; dh or u NaN reaches its row of dx and column of dw only.
    x, w = rnd(300, 64, BF16, 30), rnd(80, 64, BF16, 31)
    dh, pre = rnd(300, 40, BF16, 32), rnd(300, 80, BF16, 33)
    pre[7, 3] = float("inf")
    dh[11, 5] = float("nan")
    dx, dw, db = oz.gated_linear_backward(dh, x, w, pre)
    bad = torch.zeros(300, dtype=torch.bool, device=DEV)
    bad[7] = bad[11] = True
    assert torch.equal(~torch.isfinite(dx).all(1), bad)
    rows = torch.zeros(80, dtype=torch.bool, device=DEV)
    rows[43] = rows[5] = rows[45] = True  # u's gradient of column 3 is infinite, both of column 5 are NaN
    assert torch.equal(~torch.isfinite(dw).all(1), rows) and torch.equal(~torch.isfinite(db), rows)


def test_repeats_bit_for_bit_on_streams_and_in_graphs(oz):
    x, w, b = rnd(600, 256, BF16, 50), rnd(1200, 256, BF16, 51, 0.06), rnd(1, 1200, BF16, 52)[0]
    dh = rnd(600, 600, BF16, 53)

    def step(stream=None):
        h, pre = oz.gated_linear(x, w, b, save_pre=True, stream=stream)
        return (h, pre) + oz.gated_linear_backward(dh, x, w, pre, stream=stream)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there, here = step(side), step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(2):
        graph.replay()
    for got in (there, here, held):
        assert all(torch.equal(g, v) for g, v in zip(got, want))
