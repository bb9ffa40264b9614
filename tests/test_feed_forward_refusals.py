"""What the calls of the feed-forward operators refuse, each by the words of its own check.  (On host tensors a call that no
check refuses ends at the last one, that they lie on the GPU.)"""

import pytest

torch = pytest.importorskip("torch")

B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ON_GPU = "expected CUDA tensors"


@pytest.fixture(scope="module")
def oz():
    import ozaki_ii_fp64_gb300 as oz
    oz.load()
    return oz


def z(*shape, dtype=B16):
    return torch.zeros(*shape, dtype=dtype)


X, W, B, PRE, DH = z(2, 4), z(6, 4), z(6), z(2, 6), z(2, 3)

GATED = [
    (dict(), ON_GPU), (dict(bias=B), ON_GPU), (dict(out=z(2, 3)), ON_GPU),
    (dict(x=X.float(), w=W.float()), "bfloat16 or float16"), (dict(x=X[0]), "x: expected a 2-D tensor"),
    (dict(w=W[:5]), "an even number of rows"), (dict(w=W.half()), "w: expected a 6 x 4 matrix of BFloat16"),
    (dict(w=W[:, :3]), "w: expected a 6 x 4 matrix"), (dict(x=z(4, 2).t()), "x: expected a row-major matrix"),
    (dict(x=z(2, 8)[:, ::2]), "x: expected a row-major matrix"), (dict(w=z(4, 6).t()), "w: expected a row-major matrix"),
    (dict(w=z(1, 4).expand(6, 4)), "w: expected a row-major matrix"),
    (dict(bias=z(3)), "bias: expected a dense vector of 6 BFloat16"), (dict(bias=z(1, 6)), "bias: expected a dense vector"),
    (dict(bias=B.float()), "bias: expected a dense vector"), (dict(bias=z(12)[::2]), "bias: expected a dense vector"),
    (dict(bias=3), "bias: expected a tensor"), (dict(x=None), "x: expected a tensor"), (dict(w=[1]), "w: expected a tensor"),
    (dict(activation="tanh"), "activation"), (dict(out=z(2, 6)), "out: expected a 2 x 3 matrix"),
    (dict(out=z(2, 3, dtype=F32)), "out: expected a 2 x 3 matrix of BFloat16"),
    (dict(out=z(3, 2).t()), "out: expected a row-major matrix"),
]


@pytest.mark.parametrize("change, words", GATED)
def test_gated_linear(oz, change, words):
    call = dict(x=X, w=W)
    call.update(change)
    with pytest.raises(ValueError, match=words):
        oz.gated_linear(**call)


BACKWARD = [
    (dict(), ON_GPU), (dict(x_grad=False), ON_GPU), (dict(pre=None), "pre: expected a tensor"),
    (dict(pre=DH), "pre: expected a 2 x 6 matrix"), (dict(pre=PRE.half()), "pre: expected a 2 x 6 matrix of BFloat16"),
    (dict(pre=z(6, 2).t()), "pre: expected a row-major matrix"), (dict(dh=PRE), "dh: expected a 2 x 3 matrix"),
    (dict(dh=DH.float()), "dh: expected a 2 x 3 matrix of BFloat16"), (dict(dh=z(3, 3)), "dh: expected a 2 x 3 matrix"),
    (dict(dh=z(3).expand(2, 3)), "dh: expected a row-major matrix"), (dict(w=W[:5]), "an even number of rows"),
    (dict(x=X[:, :3]), "w: expected a 6 x 3 matrix"), (dict(activation=None), "activation"),
]


@pytest.mark.parametrize("change, words", BACKWARD)
def test_gated_linear_backward(oz, change, words):
    call = dict(dh=DH, x=X, w=W, pre=PRE)
    call.update(change)
    with pytest.raises(ValueError, match=words):
        oz.gated_linear_backward(**call)


def mx(oz, rows, cols):
    return oz.MXMatrix.empty(rows, cols, device="cpu")


QUANTIZE = [
    (lambda oz: dict(x=X), ON_GPU), (lambda oz: dict(x=X.half()), ON_GPU), (lambda oz: dict(x=X.float()), ON_GPU),
    (lambda oz: dict(x=X, out=mx(oz, 2, 4)), ON_GPU),
    (lambda oz: dict(x=X.double()), "expected bfloat16, float16 or float32, got Double"),
    (lambda oz: dict(x=X.int()), "expected bfloat16, float16 or float32, got Int"),
    (lambda oz: dict(x=X[0]), "x: expected a 2-D tensor"), (lambda oz: dict(x=3), "x: expected a tensor"),
    (lambda oz: dict(x=z(4, 2).t()), "x: expected a row-major matrix"),
    (lambda oz: dict(x=X, out=mx(oz, 3, 4)), "out: expected an MXMatrix of x's size"),
    (lambda oz: dict(x=X, out=X), "out: expected an MXMatrix"),
    (lambda oz: dict(x=X, out=oz.MXMatrix(mx(oz, 200, 4).data, 2, 4)), "out: expected a dense vector of 1280 Byte"),
    (lambda oz: dict(x=X, out=oz.MXMatrix(mx(oz, 2, 4).data.float(), 2, 4)), "out: expected a dense vector of 1280 Byte"),
]


@pytest.mark.parametrize("case", range(len(QUANTIZE)))
def test_mx_quantize(oz, case):
    make, words = QUANTIZE[case]
    with pytest.raises(ValueError, match=words):
        oz.mx_quantize(**make(oz))


DEQUANTIZE = [
    (lambda oz: dict(q=mx(oz, 2, 4)), ON_GPU), (lambda oz: dict(q=mx(oz, 2, 4), dtype=F32), ON_GPU),
    (lambda oz: dict(q=mx(oz, 2, 4), out=z(2, 4, dtype=F16)), ON_GPU), (lambda oz: dict(q=X), "q: expected an MXMatrix"),
    (lambda oz: dict(q=mx(oz, 2, 4), dtype=torch.float64), "dtype: expected one of"),
    (lambda oz: dict(q=mx(oz, 2, 4), out=z(2, 4).double()), "dtype: expected one of"),
    (lambda oz: dict(q=mx(oz, 2, 4), out=z(2, 5)), "out: expected a 2 x 4 matrix"),
    (lambda oz: dict(q=mx(oz, 2, 4), out=z(4, 2).t()), "out: expected a row-major matrix"),
    (lambda oz: dict(q=mx(oz, 2, 4), dtype=F16, out=z(2, 4)), "out: expected a matrix of Half"),
    (lambda oz: dict(q=oz.MXMatrix(mx(oz, 2, 4).data[1:], 2, 4)), "q: expected a dense vector of 1280 Byte"),
    (lambda oz: dict(q=oz.MXMatrix(mx(oz, 2, 4).data.view(2, 640), 2, 4)), "q: expected a dense vector of 1280 Byte"),
    (lambda oz: dict(q=oz.MXMatrix(torch.zeros(1284, dtype=torch.uint8)[4:], 2, 4)), "q: not on a 16-byte boundary"),
    (lambda oz: dict(q=oz.MXMatrix(mx(oz, 2, 4).data, -1, 4)), "sizes: out of range"),
]


@pytest.mark.parametrize("case", range(len(DEQUANTIZE)))
def test_mx_dequantize(oz, case):
    make, words = DEQUANTIZE[case]
    with pytest.raises(ValueError, match=words):
        oz.mx_dequantize(**make(oz))


LINEAR = [
    (lambda oz: dict(), ON_GPU), (lambda oz: dict(bias=z(3)), ON_GPU), (lambda oz: dict(residual=DH), ON_GPU),
    (lambda oz: dict(times=DH), ON_GPU), (lambda oz: dict(out=DH), ON_GPU), (lambda oz: dict(residual=DH, out=DH), ON_GPU),
    (lambda oz: dict(x=X), "x: expected an MXMatrix"), (lambda oz: dict(w=W), "w: expected an MXMatrix"),
    (lambda oz: dict(w=mx(oz, 3, 5)), "inner dimensions differ"),
    (lambda oz: dict(x=oz.MXMatrix(mx(oz, 2, 4).data, 200, 4)), "x: expected a dense vector of"),
    (lambda oz: dict(w=oz.MXMatrix(mx(oz, 2, 4).data, 200, 4)), "w: expected a dense vector of"),
    (lambda oz: dict(dtype=F32), "dtype: expected one of"), (lambda oz: dict(bias=z(3, dtype=F32)), "dtype: expected one of"),
    (lambda oz: dict(bias=z(4)), "bias: expected a dense vector of 3 BFloat16"),
    (lambda oz: dict(bias=z(3), dtype=F16), "bias: expected Half"),
    (lambda oz: dict(residual=X), "residual: expected a 2 x 3 matrix"), (lambda oz: dict(times=X), "times: expected a 2 x 3 matrix"),
    (lambda oz: dict(residual=DH, times=DH), "times: expected no residual beside it"),
    (lambda oz: dict(residual=DH, dtype=F16), "residual: expected Half"), (lambda oz: dict(times=DH, dtype=F16), "times: expected Half"),
    (lambda oz: dict(residual=DH, bias=z(3, dtype=F16)), "bias: expected a dense vector of 3 BFloat16"),
    (lambda oz: dict(out=X), "out: expected a 2 x 3 matrix"), (lambda oz: dict(out=DH, dtype=F16), "out: expected Half"),
    (lambda oz: dict(residual=DH.half(), out=DH), "residual: expected a 2 x 3 matrix of BFloat16"),
    (lambda oz: dict(out=z(3, 2).t()), "out: expected a row-major matrix"), (lambda oz: dict(activation="swish"), "activation"),
]


@pytest.mark.parametrize("case", range(len(LINEAR)))
def test_mx_linear(oz, case):
    make, words = LINEAR[case]
    call = dict(x=mx(oz, 2, 4), w=mx(oz, 3, 4))
    call.update(make(oz))
    with pytest.raises(ValueError, match=words):
        oz.mx_linear(**call)


G = z(10, dtype=F32)
CLIP = [
    (dict(), ON_GPU), (dict(grads=(G, X)), ON_GPU), (dict(out=[z(10, dtype=F32)]), ON_GPU), (dict(out=(G,)), ON_GPU),
    (dict(grads=[]), "grads: expected at least one tensor"), (dict(grads=[G, 3]), "grads: expected a sequence of tensors"),
    (dict(grads=[G, None]), "grads: expected a sequence of tensors"),
    (dict(grads=[G.double()]), "grads: expected bfloat16, float16 or float32, got Double"),
    (dict(grads=[G, G.int()]), "grads: expected bfloat16, float16 or float32, got Int"),
    (dict(grads=[G[::2]]), "grads: expected dense tensors"), (dict(grads=[G[:1].expand(4)]), "grads: expected dense tensors"),
    (dict(grads=[z(4, 6)[:, :3]]), "grads: expected dense tensors"),
    (dict(grads=[G.to_sparse()]), "grads: expected dense tensors"), (dict(out=[]), "out: expected as many tensors as grads"),
    (dict(out=[G, G]), "out: expected as many tensors as grads"), (dict(out=[3]), "out: expected a sequence of tensors"),
    (dict(out=[z(9, dtype=F32)]), "out: expected tensors of the gradients' sizes, types and device"),
    (dict(out=[z(10, dtype=F16)]), "out: expected tensors of the gradients' sizes, types and device"),
    (dict(out=[G.to_sparse()]), "out: expected tensors of the gradients' sizes, types and device"),
    (dict(grads=[z(3, 4)], out=[z(4, 3).t()]), "out: expected tensors of the gradients' strides"),
    (dict(out=[z(20, dtype=F32)[::2]]), "out: expected tensors of the gradients' strides"),
]


@pytest.mark.parametrize("change, words", CLIP)
def test_clip_grad_norm(oz, change, words):
    call = dict(grads=[G], max_norm=1.0)
    call.update(change)
    with pytest.raises(ValueError, match=words):
        oz.clip_grad_norm(**call)


@pytest.mark.parametrize("call", [dict(grads=3, max_norm=1.0), dict(grads=[G], max_norm="one"), dict(grads=[G], max_norm=None),
                                  dict(grads=[G], max_norm=1.0, eps="one"), dict(grads=[G], max_norm=1.0, out=3)])
def test_clip_grad_norm_of_other_kinds(oz, call):
    with pytest.raises(TypeError):
        oz.clip_grad_norm(**call)


@pytest.mark.parametrize("rows, cols", [(-1, 4), (4, -1), ((1 << 26) + 1, 4), (4, (1 << 26) + 1)])
def test_mx_matrix_sizes(oz, rows, cols):
    with pytest.raises(ValueError, match="expected from 0 to 2\\^26 rows and columns"):
        oz.MXMatrix.empty(rows, cols, device="cpu")


def test_mx_quantize_into_nothing_of_a_kind(oz):
    with pytest.raises(ValueError, match="x: expected a tensor"):
        oz.mx_quantize(3, out=mx(oz, 2, 4))
