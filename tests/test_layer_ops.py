"""The layer operators' references against differences, and their refusals, which need no GPU: argument checks run on
the host before any CUDA call."""

import pytest

from layer_reference import act64, linear64, linear_backward64, norm64, norm_backward64

torch = pytest.importorskip("torch")

FAKE = 0x10000  # non-null, 256-byte aligned; never dereferenced
NULL = None
BF16, F16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def oz():
    import ozaki_ii_fp64_gb300 as oz
    oz.load()
    return oz


# ---------------------------------------------------------- the references' gradients against differences

def _difference(f, x, v, h=1e-5):
    return float((f(x + h * v) - f(x - h * v)) / (2 * h))


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=torch.float64)


@pytest.fixture()
def as_float64(monkeypatch):
    # The references take their rounding bounds from the operands' type; here only the values matter.
    import layer_reference
    monkeypatch.setitem(layer_reference.U, torch.float64, 0.0)
    monkeypatch.setitem(layer_reference.TINY, torch.float64, 0.0)


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu", "relu"])
def test_linear_gradient_formulas_against_differences(as_float64, act):
    gen = torch.Generator().manual_seed(3)
    x, w, b, dy = _rand(gen, 5, 7), _rand(gen, 6, 7), _rand(gen, 6), _rand(gen, 5, 6)
    z = x @ w.t() + b
    assert float(z.abs().min()) > 1e-3  # relu's corner is out of the differences' reach
    (dx, dw, db), _ = linear_backward64(dy, x, w, z, act)
    for grad, at, f in ((dx, x, lambda t: (act64(t @ w.t() + b, act) * dy).sum()),
                        (dw, w, lambda t: (act64(x @ t.t() + b, act) * dy).sum()),
                        (db, b, lambda t: (act64(x @ w.t() + t, act) * dy).sum())):
        v = _rand(gen, *at.shape)
        # Central differences: h^2 f'''/6 and rounding 2^-52 |f| / h, both below 1e-8 here.
        assert abs(_difference(f, at, v) - float((grad * v).sum())) < 1e-6


def test_norm_gradient_formulas_against_differences(as_float64):
    gen = torch.Generator().manual_seed(4)
    x, w, b, dy = _rand(gen, 4, 9), _rand(gen, 9), _rand(gen, 9), _rand(gen, 4, 9)
    (_, mean, rstd), _ = norm64(x, w, b)
    (dx, dw, db), _ = norm_backward64(dy, x, mean, rstd, w)
    for grad, at, f in ((dx, x, lambda t: (norm64(t, w, b)[0][0] * dy).sum()),
                        (dw, w, lambda t: (norm64(x, t, b)[0][0] * dy).sum()),
                        (db, b, lambda t: (norm64(x, w, t)[0][0] * dy).sum())):
        v = _rand(gen, *at.shape)
        assert abs(_difference(f, at, v) - float((grad * v).sum())) < 1e-6


def test_reference_linear_is_the_formula(as_float64):
    gen = torch.Generator().manual_seed(5)
    x, w, b, r = _rand(gen, 3, 4), _rand(gen, 2, 4), _rand(gen, 2), _rand(gen, 3, 2)
    y, _, z, _ = linear64(x, w, b, r, "gelu")
    assert torch.allclose(z, torch.nn.functional.linear(x, w, b), rtol=1e-13, atol=1e-13)
    assert torch.allclose(y, torch.nn.functional.gelu(z) + r, rtol=1e-12, atol=1e-12)


# ------------------------------------------------------------------------------------------ refusals

def _linear(oz, m=4, n=4, k=8, type=BF16, X=FAKE, ldx=8, W=FAKE, ldw=8, bias=FAKE, R=NULL, ldr=4, act=0, pre=NULL,
            ldpre=4, Y=FAKE, ldy=4, ws=FAKE, nbytes=1 << 30):
    return oz.ozemu_linear(m, n, k, type, X, ldx, W, ldw, bias, R, ldr, act, pre, ldpre, Y, ldy, ws, nbytes, NULL)


def _linear_backward(oz, m=4, n=4, k=8, type=BF16, dY=FAKE, lddy=4, X=FAKE, ldx=8, W=FAKE, ldw=8, act=2, pre=FAKE,
                     ldpre=4, dX=FAKE, lddx=8, dW=FAKE, lddw=8, db=FAKE, ws=FAKE, nbytes=1 << 30):
    return oz.ozemu_linear_backward(m, n, k, type, dY, lddy, X, ldx, W, ldw, act, pre, ldpre, dX, lddx, dW, lddw, db,
                                    ws, nbytes, NULL)


def _norm(oz, rows=4, cols=8, type=BF16, X=FAKE, ldx=8, ptype=BF16, w=FAKE, b=FAKE, eps=1e-5, Y=FAKE, ldy=8,
          mean=NULL, rstd=NULL):
    return oz.ozemu_layer_norm(rows, cols, type, X, ldx, ptype, w, b, eps, Y, ldy, mean, rstd, NULL)


def _norm_backward(oz, rows=4, cols=8, type=BF16, dY=FAKE, lddy=8, X=FAKE, ldx=8, ptype=F32, w=FAKE, mean=FAKE,
                   rstd=FAKE, dR=NULL, lddr=8, dX=FAKE, lddx=8, dw=FAKE, db=FAKE, ws=FAKE, nbytes=1 << 30):
    return oz.ozemu_layer_norm_backward(rows, cols, type, dY, lddy, X, ldx, ptype, w, mean, rstd, dR, lddr, dX, lddx,
                                        dw, db, ws, nbytes, NULL)


@pytest.mark.parametrize("call, bad", [
    (_linear, dict(m=(1 << 26) + 1)), (_linear, dict(k=(1 << 26) + 1, ldx=1 << 27, ldw=1 << 27)),
    (_norm, dict(rows=(1 << 31) - 1)), (_norm, dict(cols=(1 << 31) - 1, ldx=(1 << 31) - 1, ldy=(1 << 31) - 1)),
    (_linear, dict(m=-1)), (_linear, dict(n=-1)), (_linear, dict(k=-1)),
    (_linear, dict(type=F32)), (_linear, dict(type=3)), (_linear, dict(type=-1)),
    (_linear, dict(act=5)), (_linear, dict(act=-1)),
    (_linear, dict(ldx=7)), (_linear, dict(ldw=7)), (_linear, dict(ldy=3)),
    (_linear, dict(R=FAKE, ldr=3)), (_linear, dict(pre=FAKE, ldpre=3)),
    (_linear, dict(X=NULL)), (_linear, dict(W=NULL)), (_linear, dict(Y=NULL)),
    (_linear, dict(X=FAKE + 1)), (_linear, dict(W=FAKE + 1)), (_linear, dict(bias=FAKE + 1)),
    (_linear, dict(R=FAKE + 1)), (_linear, dict(pre=FAKE + 1)), (_linear, dict(Y=FAKE + 1)),
    (_linear_backward, dict(m=-1)), (_linear_backward, dict(type=F32)), (_linear_backward, dict(act=9)),
    (_linear_backward, dict(dY=NULL)), (_linear_backward, dict(lddy=3)), (_linear_backward, dict(pre=NULL)),
    (_linear_backward, dict(ldpre=3)), (_linear_backward, dict(X=NULL)), (_linear_backward, dict(W=NULL)),
    (_linear_backward, dict(lddx=7)), (_linear_backward, dict(lddw=7)), (_linear_backward, dict(db=FAKE + 1)),
    (_linear_backward, dict(dW=FAKE + 1)), (_linear_backward, dict(ws=FAKE + 128)),
    (_norm, dict(rows=-1)), (_norm, dict(cols=-1)), (_norm, dict(type=3)), (_norm, dict(ptype=F16)),
    (_norm, dict(type=F32, ptype=BF16)), (_norm, dict(eps=-1.0)), (_norm, dict(eps=float("nan"))),
    (_norm, dict(ldx=7)), (_norm, dict(ldy=7)), (_norm, dict(X=NULL)), (_norm, dict(Y=NULL)),
    (_norm, dict(X=FAKE + 1)), (_norm, dict(ptype=F32, w=FAKE + 2)), (_norm, dict(mean=FAKE + 2)),
    (_norm_backward, dict(rows=-1)), (_norm_backward, dict(ptype=F16)), (_norm_backward, dict(dY=NULL)),
    (_norm_backward, dict(mean=NULL)), (_norm_backward, dict(rstd=NULL)), (_norm_backward, dict(dX=NULL)),
    (_norm_backward, dict(lddx=7)), (_norm_backward, dict(dR=FAKE, lddr=7)), (_norm_backward, dict(dw=FAKE + 2)),
])
def test_invalid_arguments_rejected_on_host(oz, call, bad):
    assert call(oz, **bad) == oz.OZEMU_ERR_INVALID_ARG


def test_small_workspace_rejected_on_host(oz):
    need = oz.ozemu_linear_backward_bytes(4, 4, 8, FAKE, 4, FAKE, 8, FAKE, 8, 2)
    assert need > 0
    assert _linear_backward(oz, nbytes=need - 1) == oz.OZEMU_ERR_SCRATCH_TOO_SMALL
    assert _linear_backward(oz, ws=NULL) == oz.OZEMU_ERR_SCRATCH_TOO_SMALL


def test_empty_problems_are_noops(oz):
    assert _linear(oz, m=0, X=NULL, Y=NULL, ws=NULL, nbytes=0) == oz.OZEMU_OK
    assert _linear(oz, n=0, W=NULL, Y=NULL, bias=NULL, ws=NULL, nbytes=0) == oz.OZEMU_OK
    assert _linear_backward(oz, m=0, n=0, ws=NULL, nbytes=0) == oz.OZEMU_OK
    assert _norm(oz, rows=0, X=NULL, Y=NULL) == oz.OZEMU_OK
    assert _norm(oz, cols=0, X=NULL, Y=NULL) == oz.OZEMU_OK
    assert _norm_backward(oz, cols=0, ws=NULL, nbytes=0) == oz.OZEMU_OK


def test_workspace_queries_on_bad_arguments(oz):
    assert oz.ozemu_linear_bytes(-1, 4, 8, FAKE, 8, FAKE, 8) == 0
    assert oz.ozemu_linear_bytes(4, 4, 8, FAKE, 7, FAKE, 8) == 0
    assert oz.ozemu_linear_backward_bytes(4, 4, 8, FAKE, 3, FAKE, 8, FAKE, 8, 2) == 0
    assert oz.ozemu_linear_backward_bytes(4, 4, 8, FAKE, 4, FAKE, 8, FAKE, 8, 7) == 0
    assert oz.ozemu_layer_norm_backward_bytes(-1, 8) == 0
    assert oz.ozemu_linear_bytes((1 << 26) + 1, 4, 8, FAKE + 2, 8, FAKE, 8) == 0


def test_binding_refuses_wrong_tensors(oz):
    x, w = torch.zeros(2, 4, dtype=torch.bfloat16), torch.zeros(3, 4, dtype=torch.bfloat16)
    for bad in (lambda: oz.linear(x, w),                                        # not on the GPU
                lambda: oz.linear(x.float(), w.float()),                        # no 32-bit products
                lambda: oz.linear(x, w.half()),
                lambda: oz.linear(x, w[:, :3]),
                lambda: oz.linear(x, w, torch.zeros(2, dtype=torch.bfloat16)),
                lambda: oz.linear(x, w, residual=torch.zeros(2, 2, dtype=torch.bfloat16)),
                lambda: oz.linear(x, w, activation="tanh"),
                lambda: oz.linear(x.t().contiguous().t(), w),                   # column-major
                lambda: oz.linear(x[:1].expand(2, 4), w),                       # broadcast rows
                lambda: oz.linear_backward(torch.zeros(2, 3, dtype=torch.bfloat16), x, w, activation="gelu"),
                lambda: oz.layer_norm(x.double()),
                lambda: oz.layer_norm(x, torch.zeros(4, dtype=torch.float16)),
                lambda: oz.layer_norm(x, torch.zeros(5, dtype=torch.bfloat16)),
                lambda: oz.layer_norm(x, torch.zeros(4), torch.zeros(4, dtype=torch.bfloat16)),
                lambda: oz.layer_norm_backward(x, x, torch.zeros(2).double(), torch.zeros(2)),
                lambda: oz.layer_norm(x[0])):
        with pytest.raises(ValueError):
            bad()
