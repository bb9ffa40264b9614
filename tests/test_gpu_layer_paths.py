"""The layer operators' paths that only larger problems take, against the 64-bit references: the norms' rings at many
rows (any alignment, in place, unaligned parameters, slots used again), and the product's accumulators used again."""

import pytest

from layer_reference import linear64, linear_backward64, norm64, norm_backward64, worst

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


def rnd(rows, cols, dtype, seed, scale=1.0, shift=0.0, pad=0, offset=0):
    """A rows x cols matrix with leading dimension cols + pad, `offset` elements into its memory, NaN around it."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ld = cols + pad
    buf = torch.full((rows * ld + offset + 8,), float("nan"), dtype=dtype, device=DEV)
    t = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    t.copy_(torch.randn(rows, cols, generator=gen, device=DEV) * scale + shift)
    return t


def vec(n, dtype, seed, offset=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(n + offset, generator=gen, device=DEV).to(dtype)[offset:]


def outside(t):
    """The bits of t's memory with t itself blanked."""
    c = t._base.clone()
    torch.as_strided(c, t.shape, t.stride(), t.storage_offset()).zero_()
    return c.view(torch.int32 if t.dtype == F32 else torch.int16)


# Rows that start anywhere, more than one SM's groups take at once, up to several turns of their slots; one shape for
# each number of threads and elements to a row, widths at the edges of what a thread count takes.
ANY_ROWS = [(5200, 131, 3, 0), (20000, 33, 0, 1), (6000, 512, 1, 0), (1300, 1025, 0, 0), (2600, 2047, 2, 5),
            (1000, 3001, 3, 1), (4000, 4096, 0, 1), (1021, 5003, 3, 0), (1500, 8191, 1, 3), (400, 9001, 0, 7),
            (700, 16383, 5, 0), (200, 17001, 0, 0), (330, 30001, 0, 1)]


@pytest.mark.parametrize("dtype, wdtype", [(BF16, BF16), (F16, F32), (F32, F32)], ids=str)
@pytest.mark.parametrize("rows, cols, pad, offset", ANY_ROWS)
def test_forward_rows_of_any_start(oz, rows, cols, pad, offset, dtype, wdtype):
    x = rnd(rows, cols, dtype, 1, 2.0, 0.5, pad, offset)
    w, b = vec(cols, wdtype, 2, offset=1), vec(cols, wdtype, 3, offset=3)
    want, bounds = norm64(x, w, b)
    got = oz.layer_norm(x, w, b, stats=True)
    for g, v, e in zip(got, want, bounds):
        assert worst(g, v, e) <= 1
    plain, e = norm64(x)
    assert worst(oz.layer_norm(x), plain[0], e[0]) <= 1
    # In place: the bits of a call whose output is laid out the same (the variant goes by alignment, its sums' order too).
    other = rnd(rows, cols, dtype, 20, pad=pad, offset=offset)
    oz.layer_norm(x, w, b, out=other)
    before = outside(x)
    assert oz.layer_norm(x, w, b, out=x) is x
    assert torch.equal(x, other) and torch.equal(outside(x), before)
    assert worst(x, want[0], bounds[0]) <= 1


# Aligned rows, each thread count of the ring, five turns and more of its slots.
@pytest.mark.parametrize("dtype, wdtype", [(BF16, BF16), (F16, F32), (F32, F32)], ids=str)
@pytest.mark.parametrize("rows, cols", [(19000, 1000), (4700, 2048), (4600, 4096), (2300, 8184), (800, 16384), (800, 32768)])
def test_forward_aligned_rows(oz, rows, cols, dtype, wdtype):
    x, w, b = rnd(rows, cols, dtype, 4, 2.0, 0.5), vec(cols, wdtype, 5), vec(cols, wdtype, 6)
    want, bounds = norm64(x, w, b)
    got = oz.layer_norm(x, w, b, stats=True)
    for g, v, e in zip(got, want, bounds):
        assert worst(g, v, e) <= 1
    assert oz.layer_norm(x, w, b, out=x) is x and torch.equal(x, got[0])


# Five turns and more of each group's slots, aligned, of exactly the threads' columns, and odd.
@pytest.mark.parametrize("dtype, wdtype", [(BF16, F32), (F16, F16), (F32, F32)], ids=str)
@pytest.mark.parametrize("rows, cols, pad, offset", [
    (25000, 248, 0, 0), (25000, 251, 2, 1), (3300, 2048, 0, 0), (3200, 2000, 8, 0), (3100, 2047, 0, 1), (1600, 4096, 0, 0),
    (1650, 4001, 3, 0), (800, 8192, 0, 0), (900, 8001, 0, 3), (780, 12000, 0, 0), (770, 16383, 1, 0)])
def test_backward_many_turns(oz, rows, cols, pad, offset, dtype, wdtype):
    where = dict(pad=pad, offset=offset)
    x, dy = rnd(rows, cols, dtype, 7, 2.0, 0.5, **where), rnd(rows, cols, dtype, 8, **where)
    dr, w = rnd(rows, cols, dtype, 9, **where), vec(cols, wdtype, 10, offset=offset)
    (_, mean, rstd), _ = norm64(x)
    mean, rstd = mean.float(), rstd.float()
    for extra in (None, dr):
        want, bounds = norm_backward64(dy, x, mean, rstd, w, extra)
        for out in (None, dy if extra is None else extra):
            kept = None if out is None else out.clone()
            before = None if out is None else outside(out)
            got = oz.layer_norm_backward(dy, x, mean, rstd, w, dresidual=extra, out=out)
            for g, v, e in zip(got, want, bounds):
                assert worst(g, v, e) <= 1
            if out is not None:
                assert got[0] is out and torch.equal(outside(out), before)
                out.copy_(kept)


# Every pair of CTAs (76 of them) works on more tiles than TMEM holds accumulators, whatever width the cost model takes:
# now 256, 192, 128 and 64 columns a tile, ragged on both edges, and tiles of few columns, whose idle warps hand the
# accumulator back too.
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m, k, n", [(5000, 200, 8200), (100000, 72, 190), (100000, 100, 100), (100003, 70, 60),
                                     (100003, 64, 9), (90001, 65, 129), (40001, 33, 520)])
def test_accumulators_used_again(oz, m, k, n, dtype):
    x, w = rnd(m, k, dtype, 11), rnd(n, k, dtype, 12, k ** -0.5)
    b, r = vec(n, dtype, 13), rnd(m, n, dtype, 14)
    y, pre = oz.linear(x, w, b, r, activation="silu", save_pre=True)
    ref, tol, z, tolz = linear64(x, w, b, r, "silu")
    assert worst(y, ref, tol) <= 1 and worst(pre, z, tolz) <= 1
    del z, tolz, pre
    ref, tol, _, _ = linear64(x, w)
    assert worst(oz.linear(x, w), ref, tol) <= 1


# The same for the gradients: dx and dw in one launch, of equal and of different widths, either product first, and in
# launches of their own.
@pytest.mark.parametrize("m, k, n", [(300, 4100, 8200), (1000, 8200, 520), (9000, 8200, 100), (9000, 520, 2100),
                                     (9000, 8200, 300), (100000, 260, 120), (20000, 2100, 260)])
def test_gradients_accumulators_used_again(oz, m, k, n):
    x, w = rnd(m, k, BF16, 15), rnd(n, k, BF16, 16, k ** -0.5)
    dy, pre = rnd(m, n, BF16, 17), rnd(m, n, BF16, 18)
    for act in ("none", "silu"):
        got = oz.linear_backward(dy, x, w, pre, activation=act)
        want, bounds = linear_backward64(dy, x, w, pre, act)
        for g, v, e in zip(got, want, bounds):
            assert worst(g, v, e) <= 1
