"""Clipping of gradients whose squares leave fp32's range where the norm does not."""

import math

import pytest

from layer_reference import EPS, TINY, U, worst

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
# A thread's squares and their sum are a chain of 40 fp32 roundings at most, each half of EPS and all of one sign at worst;
# the norm has half of their sum, and its own rounding.
NORM = 11 * EPS


@pytest.fixture(scope="module")
def oz():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ozaki_ii_fp64_gb300 as oz
    oz.load()
    return oz


def rnd(n, dtype, seed, scale):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(n, generator=gen, device=DEV, dtype=torch.float64) * scale).to(dtype)


def check(oz, grads, max_norm):
    norm64 = math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))
    limit = float(torch.tensor(max_norm, dtype=F32))  # as the call takes it
    factor = min(1.0, limit / norm64)
    norm, clipped = oz.clip_grad_norm(grads, max_norm, eps=0.0)
    assert abs(float(norm) - norm64) <= NORM * norm64 + 2.0 ** -150
    for g, c in zip(grads, clipped):
        want = g.double() * factor
        # The factor: the norm's error, a sum, a quotient (a subnormal one off by 2^-150); the product; the rounding.
        tol = (U[g.dtype] + NORM + 4 * EPS) * want.abs() + g.double().abs() * 2.0 ** -150 + TINY[g.dtype]
        assert worst(c, want, tol) <= 1


SIZES = [1, 7, 1000, 20000, 1500000]  # parts of a vector, parts of a chunk, one launch and two


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("scale", [1e18, 1e20, 1e25, 1e32, 1e-17, 1e-19, 1e-21, 1e-25, 1e-32, 1e-36])
def test_one_scale(oz, size, dtype, scale):
    check(oz, [rnd(size, dtype, 1, scale)], scale / 3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_large_element(oz, dtype):
    for size in (5, 3000, 1500000):
        for at in (0, size // 2, size - 1):
            g = torch.ones(size, dtype=dtype, device=DEV)
            g[at] = 2.0 ** 70
            check(oz, [g, rnd(100, F32, 2, 1.0)], 1.0)


def test_scales_side_by_side(oz):
    # Chunks of every size in one list: the large ones make the norm, and each by itself.
    grads = [rnd(9000, F32, i, 10.0 ** e) for i, e in enumerate((-30, -22, -5, 0, 4, 19, 28))]
    check(oz, grads, 1e20)
    for g in grads:
        check(oz, [g[1:], g[:1]], 1e-10)
    check(oz, [torch.cat(grads), rnd(33, BF16, 9, 1e-30)], 1.0)


def test_subnormal_gradients(oz):
    check(oz, [rnd(5000, F32, 3, 1e-40)], 1e-39)
    g = torch.full((1 << 16,), 2.0 ** -149, device=DEV)
    norm, (c,) = oz.clip_grad_norm([g], 1.0, eps=0.0)
    assert float(norm) == 2.0 ** -141 and torch.equal(c, g)


def test_a_norm_beyond_the_type(oz):
    # 1024 elements of 2^125: the norm is 2^130.
    g = torch.full((1024,), 2.0 ** 125, device=DEV)
    norm, (c,) = oz.clip_grad_norm([g], 1.0)
    assert float(norm) == math.inf and not c.any()
