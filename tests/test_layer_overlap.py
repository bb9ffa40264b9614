"""An output given to a layer operator shares no element with an input, except the one that it may be.  Checked before
anything is asked of a GPU: a call that passes the check is refused for its CPU tensors."""

import random

import pytest

torch = pytest.importorskip("torch")

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def oz():
    import ozaki_ii_fp64_gb300 as oz
    oz.load()
    return oz


def refused(call):
    with pytest.raises(ValueError) as e:
        call()
    text = str(e.value)
    assert "overlaps" in text or "CUDA" in text
    return "overlaps" in text


def view(buf, rows, cols, ld, at):
    return torch.as_strided(buf, (rows, cols), (ld, 1), at)


def cells(rows, cols, ld, at):
    return {at + i * ld + j for i in range(rows) for j in range(cols)}


def test_linear(oz):
    buf = torch.zeros(4000, dtype=BF16)
    x, w, r = view(buf, 8, 16, 16, 0), torch.zeros(16, 16, dtype=BF16), torch.zeros(8, 16, dtype=BF16)
    b = torch.zeros(16, dtype=BF16)
    assert refused(lambda: oz.linear(x, w, out=x))
    assert refused(lambda: oz.linear(x, w, out=view(buf, 8, 16, 16, 127)))
    assert not refused(lambda: oz.linear(x, w, out=view(buf, 8, 16, 16, 128)))
    assert refused(lambda: oz.linear(x, w, out=w[:8]))
    assert not refused(lambda: oz.linear(x, w, b, r, out=r))
    assert refused(lambda: oz.linear(x, w, b, view(buf, 8, 16, 16, 1000), out=view(buf, 8, 16, 16, 1001)))
    assert refused(lambda: oz.linear(x, w, b, view(buf, 8, 16, 16, 1000), out=view(buf, 8, 16, 32, 1000)))
    assert refused(lambda: oz.linear(x, w, view(buf, 1, 16, 16, 1100)[0], out=view(buf, 8, 16, 16, 1000)))
    assert not refused(lambda: oz.linear(x, w, b, r))  # nothing given


def test_norms(oz):
    buf = torch.zeros(4000, dtype=BF16)
    x, dy = view(buf, 8, 16, 16, 0), view(buf, 8, 16, 16, 128)
    w = view(buf, 1, 16, 16, 256)[0]
    mean, rstd = torch.zeros(8), torch.ones(8)
    assert not refused(lambda: oz.layer_norm(x, w, out=x))
    assert not refused(lambda: oz.layer_norm(x, w, out=dy))
    assert refused(lambda: oz.layer_norm(x, w, out=view(buf, 8, 16, 16, 8)))
    assert refused(lambda: oz.layer_norm(x, w, out=view(buf, 8, 16, 16, 144)))
    for same in (x, dy):
        assert not refused(lambda same=same: oz.layer_norm_backward(dy, x, mean, rstd, w, out=same))
    assert refused(lambda: oz.layer_norm_backward(dy, x, mean, rstd, w, out=view(buf, 8, 16, 16, 120)))
    assert refused(lambda: oz.layer_norm_backward(dy, x, mean, rstd, w, out=view(buf, 8, 16, 16, 260)))


def test_statistics(oz):
    pool = torch.zeros(400)
    x, dy = torch.zeros(8, 16), torch.zeros(8, 16)
    out = torch.as_strided(pool, (8, 16), (16, 1), 0)
    inside, outside = pool[100:108], pool[128:136]
    good = torch.zeros(8)
    assert refused(lambda: oz.layer_norm_backward(dy, x, inside, good, out=out))
    assert refused(lambda: oz.layer_norm_backward(dy, x, good, inside, out=out))
    assert not refused(lambda: oz.layer_norm_backward(dy, x, outside, good, out=out))


def test_against_the_sets_of_elements(oz):
    # Matrices inside each other's memory: columns of one buffer, rows of different lengths.
    rng = random.Random(5)
    buf = torch.zeros(600, dtype=BF16)
    seen = [0, 0]
    for _ in range(3000):
        rows, cols = rng.randint(1, 6), rng.randint(1, 9)
        ld_x = cols + rng.choice((0, 1, 3, 10, 17))
        ld_o = rng.choice((ld_x, cols + rng.choice((0, 2, 5, 11, 24))))
        at_x, at_o = rng.randint(0, 120), rng.randint(0, 120)
        x, out = view(buf, rows, cols, ld_x, at_x), view(buf, rows, cols, ld_o, at_o)
        same = at_x == at_o and (ld_x == ld_o or rows == 1)
        want = not same and bool(cells(rows, cols, ld_x, at_x) & cells(rows, cols, ld_o, at_o))
        assert refused(lambda: oz.layer_norm(x, out=out)) == want
        seen[want] += 1
    assert min(seen) > 500
