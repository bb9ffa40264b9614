"""The feed-forward operators where an element's number passes 2^31, on rows picked from the start, the border and the end,
and what their calls say of inputs that require a gradient."""

import pytest

import mx_reference as ref
from layer_reference import EPS, act64, linear64, worst

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def oz():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ozaki_ii_fp64_gb300 as oz
    oz.load()
    return oz


@pytest.fixture(autouse=True)
def memory(oz):
    yield
    assert oz.get_status() == oz.OZEMU_OK
    torch.cuda.empty_cache()


def rnd(rows, cols, seed, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.empty(rows, cols, dtype=BF16, device=DEV)
    for i in range(0, rows, 8192):  # no large temporaries
        part = t[i:i + 8192]
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV).mul_(scale))
    return t


def picked(rows, cols):
    border = 2 ** 31 // cols
    return torch.tensor([0, border - 1, border, border + 1, rows - 1], device=DEV)


def test_quantize(oz):
    rows, cols = 66000, 33000
    x = rnd(rows, cols, 1)
    i = picked(rows, cols)
    q = oz.mx_quantize(x)
    codes, scales = ref.quantize(x[i].double().cpu().numpy())
    want = torch.from_numpy(ref.values(codes, scales)[:, :cols]).to(DEV)
    assert torch.equal(oz.mx_dequantize(q)[i].double(), want)
    few = oz.mx_quantize(x[i].contiguous())
    assert torch.equal(q.codes[i], few.codes)


@pytest.mark.parametrize("n", [16512, 16501])  # rows on boundaries, and on none
def test_product(oz, n):
    m, k = 131000, 64
    x, w, b = rnd(m, k, 2), rnd(n, k, 3, 0.125), rnd(1, n, 4)[0]
    xq, wq = oz.mx_quantize(x), oz.mx_quantize(w)
    y = oz.mx_linear(xq, wq, b, activation="silu")
    i = picked(m, n)
    want, tol, _, _ = linear64(oz.mx_dequantize(xq)[i], oz.mx_dequantize(wq), b, None, "silu")
    assert worst(y[i], want, tol) <= 1


@pytest.mark.parametrize("n", [16512, 16501])
def test_gated(oz, n):
    m, k = 66000, 64
    x, w = rnd(m, k, 5), rnd(2 * n, k, 6, 0.125)
    h, pre = oz.gated_linear(x, w, save_pre=True)
    i = torch.cat((picked(m, 2 * n), picked(m, n)[-1:]))
    _, _, z, tolz = linear64(x[i], w)
    assert worst(pre[i], z, tolz) <= 1
    gate, up = z.chunk(2, 1)
    want = act64(gate, "silu") * up
    # From sums within tolz of the formula's (their rounding to 16 bits is in it and more than covers the activation's).
    eg, eu = tolz.chunk(2, 1)
    tol = 1.2 * eg * up.abs() + (act64(gate, "silu").abs() + 1.2 * eg) * eu + 2.0 ** -7 * want.abs()
    assert worst(h[i], want, tol) <= 1
    # dx of a row is its own, and the gradients' sums are those of halves.
    dh = rnd(m, n, 7, 0.125)
    dx, dw, db = oz.gated_linear_backward(dh, x, w, pre)
    j = i.sort().values
    few = oz.gated_linear_backward(dh[j].contiguous(), x[j].contiguous(), w, pre[j].contiguous(), w_grad=False,
                                   bias_grad=False)[0]
    # Other tiles, other orders of the same sums: within two roundings and the sums' own errors.
    scale = dx[j].double().abs().amax()
    assert float((dx[j].double() - few.double()).abs().amax()) <= 2.0 ** -7 * float(scale)
    del few, dx
    half = m // 2
    parts = [oz.gated_linear_backward(dh[s], x[s], w, pre[s], x_grad=False) for s in (slice(0, half), slice(half, m))]
    for got, a, c in ((dw, parts[0][1], parts[1][1]), (db, parts[0][2], parts[1][2])):
        both = a.double() + c.double()
        bound = 2.0 ** -8 * (a.double().abs() + c.double().abs() + got.double().abs())
        # The halves' and the whole's roundings, and fp32 sums of 66000 terms of a few units at most.
        assert worst(got, both, bound + 66000 * EPS * 8) <= 1


def test_clip(oz):
    g = torch.empty(2 ** 31 + 12345, dtype=BF16, device=DEV)
    for i in range(0, g.numel(), 1 << 28):
        g[i:i + (1 << 28)].fill_(1.0 / 64)
    g[-1] = 512.0
    expect = (512.0 ** 2 + (g.numel() - 1) / 4096) ** 0.5
    norm, (c,) = oz.clip_grad_norm([g], 64.0)
    assert abs(float(norm) - expect) <= 41 * EPS * expect
    factor = 64.0 / (expect + 1e-6)
    for at, value in ((0, 1.0 / 64), (2 ** 31 - 1, 1.0 / 64), (2 ** 31, 1.0 / 64), (g.numel() - 1, 512.0)):
        assert abs(float(c[at]) - value * factor) <= 2.0 ** -8 * value * factor * 1.01
    assert bool((c[:-1] == c[0]).all())


def test_inputs_that_require_a_gradient(oz):
    x, w = rnd(3, 64, 8).requires_grad_(), rnd(16, 64, 9)
    for call in (lambda: oz.gated_linear(x, w), lambda: oz.mx_quantize(x), lambda: oz.clip_grad_norm([x], 1.0),
                 lambda: oz.gated_linear_backward(rnd(3, 8, 1), x, w, rnd(3, 16, 2))):
        with pytest.warns(UserWarning, match="records no graph"):
            call()
    xq, wq = oz.mx_quantize(x.detach()), oz.mx_quantize(w)
    with pytest.warns(UserWarning, match="records no graph"):
        oz.mx_linear(xq, wq, rnd(1, 16, 3)[0].requires_grad_())
    with torch.no_grad():
        assert not oz.gated_linear(x, w).requires_grad
