"""Clipping gradients by their global norm, against 64 bits."""

import math

import pytest

from layer_reference import EPS, TINY, U, worst

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
# A thread's squares and their sum: a chain of at most 80 fp32 operations on positive values, then 64 bits; the norm has
# half of that, and its own rounding.
NORM = 41 * EPS


@pytest.fixture(scope="module")
def oz():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ozaki_ii_fp64_gb300 as oz
    oz.load()
    return oz


def rnd(shape, dtype, seed, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def check(oz, grads, max_norm, eps=1e-6, **how):
    norm64 = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    factor = min(1.0, max_norm / (norm64 + eps))
    keep = [g.clone() for g in grads]
    norm, clipped = oz.clip_grad_norm(grads, max_norm, eps, **how)
    assert norm.shape == () and norm.dtype == F32
    assert abs(float(norm) - norm64) <= NORM * norm64
    for g, c in zip(keep, clipped):
        assert c.shape == g.shape and c.dtype == g.dtype and c.stride() == g.stride()
        want = g.double() * factor
        if factor == 1.0 and norm64 * (1 + NORM) + eps < max_norm:
            assert torch.equal(c, g)
        # The factor: the norm's error, a sum and a quotient; the product; the rounding.
        tol = (U[g.dtype] + NORM + 4 * EPS) * want.abs() + TINY[g.dtype]
        assert worst(c, want, tol) <= 1
    return norm, clipped


SIZES = [(1,), (7,), (8,), (64, 3), (5, 0), (1023,), (4096, 3), (2, 3, 5, 7), (16384,), (16385,), (300, 511), (1 << 20,)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", SIZES, ids=str)
def test_one_tensor(oz, shape, dtype):
    check(oz, [rnd(shape, dtype, 1)], 0.5)


@pytest.mark.parametrize("max_norm", [0.0, 1e-3, 1.0, 1e6, float("inf")])
def test_mixed_list(oz, max_norm):
    grads = [rnd(s, t, i, 0.1) for i, (s, t) in enumerate((s, t) for s in SIZES for t in (BF16, F16, F32))]
    check(oz, grads, max_norm)
    held = [g.clone() for g in grads]
    norm, out = check(oz, grads, max_norm, out=grads)
    assert all(o is g for o, g in zip(out, grads))
    fresh = oz.clip_grad_norm(held, max_norm)
    assert torch.equal(fresh[0], norm) and all(torch.equal(a, b) for a, b in zip(fresh[1], grads))


@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 8])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_views_of_a_flat_buffer(oz, dtype, offset):
    sizes = [3, 1, 20000, 17, 8, 40000, 1, 5, 16384]
    buf = torch.full((offset + sum(sizes) + 9,), float("nan"), dtype=dtype, device=DEV)
    views, at = [], offset
    for i, n in enumerate(sizes):
        views.append(buf[at:at + n])
        views[-1].copy_(rnd((n,), dtype, i))
        at += n
    want = oz.clip_grad_norm([v.clone() for v in views], 1.0)[1]  # other alignments
    check(oz, views, 1.0)
    other = torch.full((offset + sum(sizes) + 12,), float("nan"), dtype=dtype, device=DEV)  # starts elsewhere
    outs = [o[:] for o in other[3:3 + sum(sizes)].split(sizes)]
    check(oz, views, 1.0, out=outs)
    check(oz, views, 1.0, out=views)
    assert all(torch.allclose(v.double(), w.double(), rtol=2.0 ** -7, atol=0) for v, w in zip(views, want))
    assert torch.isnan(buf[:offset]).all() and torch.isnan(buf[at:]).all()
    assert torch.isnan(other[:3]).all() and torch.isnan(other[3 + sum(sizes):]).all()


def test_dense_tensors_of_any_order(oz):
    check(oz, [rnd((30, 70), BF16, 1).t(), rnd((4, 5, 6), F32, 2).permute(2, 0, 1)], 1.0)


@pytest.mark.parametrize("count", [63, 64, 65, 256, 257, 960, 961, 2500])
def test_long_lists(oz, count):
    base = rnd((count * 8 + 100,), F32, 3)
    grads = [base[8 * i:8 * i + 1 + i % 7] for i in range(count)]
    check(oz, grads, 0.25)


def test_gradients_of_zeros_and_nothing(oz):
    norm, (a, b) = oz.clip_grad_norm([torch.zeros(100, device=DEV), torch.zeros(0, dtype=BF16, device=DEV)], 1.0)
    assert float(norm) == 0 and not a.any() and b.numel() == 0
    norm, _ = oz.clip_grad_norm([torch.zeros(0, device=DEV)], 1.0)
    assert float(norm) == 0


def test_infinities_and_nan(oz):
    g = torch.ones(1000, device=DEV)
    g[5] = float("inf")
    norm, (c, d) = oz.clip_grad_norm([g, torch.ones(10, dtype=BF16, device=DEV)], 1.0)
    assert float(norm) == math.inf and torch.isnan(c[5]) and not c[:5].any() and not d.any()
    g[5] = float("nan")
    norm, (c, d) = oz.clip_grad_norm([g, torch.ones(10, dtype=BF16, device=DEV)], 1.0)
    assert math.isnan(float(norm)) and torch.isnan(c).all() and torch.isnan(d).all()


def test_repeats_bit_for_bit_on_streams_and_in_graphs(oz):
    grads = [rnd((3000, 500), BF16, 1), rnd((77777,), F32, 2), rnd((1,), F16, 3)]
    norm, want = oz.clip_grad_norm(grads, 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there, here = oz.clip_grad_norm(grads, 1.0, stream=side), oz.clip_grad_norm(grads, 1.0)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = oz.clip_grad_norm(grads, 1.0)
    for _ in range(2):
        graph.replay()
    for got in (there, here, held):
        assert torch.equal(got[0], norm) and all(torch.equal(a, b) for a, b in zip(got[1], want))
