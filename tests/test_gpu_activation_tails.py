"""The activations and gelu's slope where their values are small: errors relative to the value, not to the argument.

z comes exactly (one product by 1).  What may differ before the one rounding to 16 bits, relative to the value: the
approximation of the normal distribution's tail (2^-20), some twelve fp32 roundings (2^-20.4), and the exponential, within
(2 + 1.2 |a|) 2^-23 of its argument a by CUDA's documentation for __expf, and |a| 2^-23 more for the argument's own
roundings: together below 2^-19 + (1 + |a|) 2^-22.
"""

import math

import pytest

from layer_reference import TINY, U, act64, slope64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def oz():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ozaki_ii_fp64_gb300 as oz
    oz.load()
    return oz


def exponent(z, act):
    """The argument of the activation's exponential."""
    if act == "gelu":
        return z * z / 2
    return z.abs() if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3).abs()


def sweep(dtype, act):
    """Every value of the type whose exponential stays below e^80, signs of both, from 2^-12 on."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32, device=DEV).to(torch.int16)
    z = bits.view(dtype)
    zd = z.double()
    keep = torch.isfinite(zd) & (zd.abs() >= 2.0 ** -12) & (exponent(zd, act) <= 80)
    return z[keep].contiguous()


def relative(z, act):
    return 2.0 ** -19 + (1 + exponent(z, act)) * 2.0 ** -22


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("layout", ["rows", "row"])  # the kernels of many and of few rows
def test_small_values(oz, act, dtype, layout):
    z = sweep(dtype, act)
    one = torch.ones(1, 1, dtype=dtype, device=DEV)
    if layout == "rows":
        y, pre = oz.linear(z[:, None], one, activation=act, save_pre=True)
    else:
        y, pre = oz.linear(one, z[:, None], activation=act, save_pre=True)
    assert torch.equal(pre.flatten(), z)
    want = act64(z.double(), act)
    u = U[dtype]
    bound = u * want.abs() + (1 + u) * relative(z.double(), act) * want.abs() + TINY[dtype]
    assert float(((y.flatten().double() - want).abs() / bound).max()) <= 1


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows", [1, 300])  # few rows, and chunks of many
def test_small_slopes_of_gelu(oz, dtype, rows):
    # The slope's two terms have opposite signs below 0: the error is relative to their magnitudes.  db of one row that
    # counts, of `rows` (the others' gradients are 0), is the slope.
    z = sweep(dtype, "gelu")
    n = z.numel()
    dy, pre = torch.zeros(rows, n, dtype=dtype, device=DEV), torch.zeros(rows, n, dtype=dtype, device=DEV)
    dy[rows // 2], pre[rows // 2] = 1, z
    x, w = torch.zeros(rows, 8, dtype=dtype, device=DEV), torch.zeros(n, 8, dtype=dtype, device=DEV)
    _, _, db = oz.linear_backward(dy, x, w, pre, activation="gelu", x_grad=False, w_grad=False)
    zd = z.double()
    want = slope64(zd, "gelu")
    phi = torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
    magnitude = 0.5 * torch.erfc(-zd / math.sqrt(2)) + zd.abs() * phi
    u = U[dtype]
    bound = u * want.abs() + (1 + u) * relative(zd, "gelu") * magnitude + TINY[dtype]
    assert float(((db.double() - want).abs() / bound).max()) <= 1
