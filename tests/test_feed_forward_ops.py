"""The gated layer, microscaled matrices and gradient clipping without a GPU: the references against differences and
against the formats' definition, refusals, and the host side with every launch of a call failing in turn."""

import ctypes
import os
import platform
import subprocess

import numpy as np
import pytest

import mx_reference
from layer_reference import act64, slope64

torch = pytest.importorskip("torch")

HERE = os.path.dirname(os.path.abspath(__file__))
FAKE = 0x10000  # non-null, 256-byte aligned; never dereferenced
NULL = None
BF16, F16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def oz():
    import ozaki_ii_fp64_gb300 as oz
    oz.load()
    return oz


# ------------------------------------------------------------------------------------------ references

@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_gated_gradient_formulas_against_differences(act):
    gen = torch.Generator().manual_seed(3)
    n = 6
    x, w, b = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((5, 7), (2 * n, 7), (2 * n,)))
    dh = torch.randn(5, n, generator=gen, dtype=torch.float64)

    def h(x, w, b):
        z = x @ w.t() + b
        return act64(z[:, :n], act) * z[:, n:]
    z = x @ w.t() + b
    assert float(z.abs().min()) > 1e-3  # relu's corner is out of the differences' reach
    dz = torch.cat((dh * z[:, n:] * slope64(z[:, :n], act), dh * act64(z[:, :n], act)), 1)
    for grad, at, f in ((dz @ w, x, lambda t: (h(t, w, b) * dh).sum()), (dz.t() @ x, w, lambda t: (h(x, t, b) * dh).sum()),
                        (dz.sum(0), b, lambda t: (h(x, w, t) * dh).sum())):
        v = torch.randn(*at.shape, generator=gen, dtype=torch.float64)
        d = float((f(at + 1e-5 * v) - f(at - 1e-5 * v)) / 2e-5)
        # Central differences: h^2 f'''/6 and rounding 2^-52 |f| / h, both below 1e-8 here.
        assert abs(d - float((grad * v).sum())) < 1e-6


def test_mx_reference_is_the_nearest_value():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 96)) * np.exp2(rng.integers(-20, 20, (50, 1)).astype(float))
    codes, scales = mx_reference.quantize(x)
    v = mx_reference.values(codes, scales)
    s = np.repeat(np.exp2(scales.astype(float) - 127), 32, axis=1)
    most = np.abs(x).reshape(50, 3, 32).max(2)
    assert np.array_equal(scales, np.floor(np.log2(most)).astype(int) - 2 + 127)
    every = np.concatenate((mx_reference.GRID, -mx_reference.GRID))
    nearest = np.abs(x[:, :, None] / s[:, :, None] - every).min(2)
    assert np.array_equal(np.abs(x / s - v / s), nearest)
    assert np.all(np.abs(x / s) < 8)


def test_mx_reference_layout():
    # Each scale at its place, each code in its half byte.
    scales = np.arange(130 * 9).reshape(130, 9) % 251
    codes = np.arange(130 * 288).reshape(130, 288) % 16
    packed, tiles = mx_reference.pack(codes, scales, 130, 270)
    assert packed.shape == (130, 144) and tiles.shape == (2, 2, 1024)
    assert packed[5, 7] == codes[5, 14] + 16 * codes[5, 15]
    assert tiles[0, 0, 0] == scales[0, 0] and tiles[0, 0, 3] == scales[0, 3] and tiles[0, 0, 512] == scales[0, 4]
    assert tiles[0, 0, 16] == scales[1, 0] and tiles[0, 0, 4] == scales[32, 0] and tiles[0, 1, 0] == scales[0, 8]
    assert tiles[1, 0, 0] == scales[128, 0] and tiles[1, 0, 32] == 127 and tiles[0, 1, 1] == 127


def test_mx_sizes(oz):
    for rows, k, codes, tiles in ((1, 1, 16, 1), (3, 32, 48, 1), (3, 33, 96, 1), (128, 256, 128 * 128, 1),
                                  (129, 257, 129 * 144, 4), (0, 5, 0, 0), (5, 0, 0, 0), (1 << 26, 1, 1 << 30, 1 << 19)):
        assert oz.ozemu_mx_code_bytes(rows, k) == codes and oz.ozemu_mx_scale_bytes(rows, k) == tiles * 1024
    for rows, k in ((-1, 5), (5, -1), ((1 << 26) + 1, 5), (5, (1 << 26) + 1)):
        assert oz.ozemu_mx_code_bytes(rows, k) == 0 and oz.ozemu_mx_scale_bytes(rows, k) == 0


# ------------------------------------------------------------------------------------------ refusals

def _gated(oz, m=4, n=4, k=8, type=BF16, X=FAKE, ldx=8, W=FAKE, ldw=8, bias=FAKE, act=4, pre=NULL, ldpre=8, H=FAKE, ldh=4,
           ws=FAKE, nbytes=1 << 30):
    return oz.ozemu_gated_linear(m, n, k, type, X, ldx, W, ldw, bias, act, pre, ldpre, H, ldh, ws, nbytes, NULL)


def _gated_backward(oz, m=4, n=4, k=8, type=BF16, dH=FAKE, lddh=4, X=FAKE, ldx=8, W=FAKE, ldw=8, act=4, pre=FAKE, ldpre=8,
                    dX=FAKE, lddx=8, dW=FAKE, lddw=8, db=FAKE, ws=FAKE, nbytes=1 << 30):
    return oz.ozemu_gated_linear_backward(m, n, k, type, dH, lddh, X, ldx, W, ldw, act, pre, ldpre, dX, lddx, dW, lddw, db,
                                          ws, nbytes, NULL)


def _quantize(oz, rows=4, k=8, type=BF16, X=FAKE, ldx=8, codes=FAKE, scales=FAKE):
    return oz.ozemu_mx_quantize(rows, k, type, X, ldx, codes, scales, NULL)


def _dequantize(oz, rows=4, k=8, type=BF16, codes=FAKE, scales=FAKE, Y=FAKE, ldy=8):
    return oz.ozemu_mx_dequantize(rows, k, type, codes, scales, Y, ldy, NULL)


def _mx_linear(oz, m=4, n=4, k=8, type=BF16, xc=FAKE, xs=FAKE, wc=FAKE, ws=FAKE, bias=FAKE, R=NULL, ldr=4, times=0, act=0,
               Y=FAKE, ldy=4):
    return oz.ozemu_mx_linear(m, n, k, type, xc, xs, wc, ws, bias, R, ldr, times, act, Y, ldy, NULL)


def _arrays(grads=(FAKE,), sizes=(10,), types=(F32,), outs=(FAKE,)):
    def array(values, kind):
        return None if values is None else (kind * max(len(values), 1))(*values)
    return (array(grads, ctypes.c_void_p), array(sizes, ctypes.c_longlong), array(types, ctypes.c_int),
            array(outs, ctypes.c_void_p))


def _clip(oz, count=1, max_norm=1.0, eps=1e-6, norm=FAKE, ws=FAKE, nbytes=1 << 20, **arrays):
    g, s, t, o = _arrays(**arrays)
    return oz.ozemu_clip_grad_norm(count, g, s, t, o, max_norm, eps, norm, ws, nbytes, NULL)


@pytest.mark.parametrize("call, bad", [
    (_gated, dict(m=-1)), (_gated, dict(n=-1)), (_gated, dict(k=-1)), (_gated, dict(n=(1 << 25) + 1)),
    (_gated, dict(m=(1 << 26) + 1)), (_gated, dict(type=F32)), (_gated, dict(act=5)), (_gated, dict(ldx=7)),
    (_gated, dict(ldw=7)), (_gated, dict(ldh=3)), (_gated, dict(pre=FAKE, ldpre=7)), (_gated, dict(X=NULL)),
    (_gated, dict(W=NULL)), (_gated, dict(H=NULL)), (_gated, dict(bias=FAKE + 1)), (_gated, dict(H=FAKE + 1)),
    (_gated_backward, dict(m=-1)), (_gated_backward, dict(type=F32)), (_gated_backward, dict(act=-1)),
    (_gated_backward, dict(dH=NULL)), (_gated_backward, dict(lddh=3)), (_gated_backward, dict(pre=NULL)),
    (_gated_backward, dict(act=0, pre=NULL)), (_gated_backward, dict(ldpre=7)), (_gated_backward, dict(X=NULL)),
    (_gated_backward, dict(W=NULL)), (_gated_backward, dict(lddx=7)), (_gated_backward, dict(lddw=7)),
    (_gated_backward, dict(db=FAKE + 1)), (_gated_backward, dict(ws=FAKE + 128)),
    (_quantize, dict(rows=-1)), (_quantize, dict(k=-1)), (_quantize, dict(rows=(1 << 26) + 1)), (_quantize, dict(type=3)),
    (_quantize, dict(X=NULL)), (_quantize, dict(ldx=7)), (_quantize, dict(type=F32, X=FAKE + 2)),
    (_quantize, dict(codes=NULL)), (_quantize, dict(scales=NULL)), (_quantize, dict(codes=FAKE + 8)),
    (_quantize, dict(scales=FAKE + 8)), (_dequantize, dict(rows=-1)), (_dequantize, dict(type=-1)),
    (_dequantize, dict(Y=NULL)), (_dequantize, dict(ldy=7)), (_dequantize, dict(codes=NULL)),
    (_dequantize, dict(scales=FAKE + 4)), (_mx_linear, dict(m=-1)), (_mx_linear, dict(k=(1 << 26) + 1)),
    (_mx_linear, dict(type=F32)), (_mx_linear, dict(act=5)), (_mx_linear, dict(xc=NULL)), (_mx_linear, dict(xs=NULL)),
    (_mx_linear, dict(wc=FAKE + 8)), (_mx_linear, dict(ws=NULL)), (_mx_linear, dict(Y=NULL)), (_mx_linear, dict(ldy=3)),
    (_mx_linear, dict(R=FAKE, ldr=3)), (_mx_linear, dict(R=FAKE + 1)), (_mx_linear, dict(bias=FAKE + 1)),
    (_clip, dict(count=-1)), (_clip, dict(grads=None)), (_clip, dict(sizes=None)), (_clip, dict(types=None)),
    (_clip, dict(outs=None)), (_clip, dict(max_norm=-1.0)), (_clip, dict(max_norm=float("nan"))), (_clip, dict(eps=-1.0)),
    (_clip, dict(eps=float("nan"))), (_clip, dict(max_norm=0.0, eps=0.0)), (_clip, dict(norm=FAKE + 2)),
    (_clip, dict(sizes=(-1,))), (_clip, dict(sizes=((1 << 40) + 1,))), (_clip, dict(types=(3,))), (_clip, dict(grads=(0,))),
    (_clip, dict(outs=(0,))), (_clip, dict(grads=(FAKE + 2,))), (_clip, dict(outs=(FAKE + 1,))),
    (_clip, dict(sizes=(1 << 30,), ws=FAKE + 8)),
])
def test_invalid_arguments_rejected_on_host(oz, call, bad):
    assert call(oz, **bad) == oz.OZEMU_ERR_INVALID_ARG


def test_small_workspaces_rejected_on_host(oz):
    need = oz.ozemu_gated_linear_backward_bytes(4, 4, 8, FAKE, 8, FAKE, 8)
    assert need > 0 and _gated_backward(oz, nbytes=need - 1) == oz.OZEMU_ERR_SCRATCH_TOO_SMALL
    assert _gated_backward(oz, ws=NULL) == oz.OZEMU_ERR_SCRATCH_TOO_SMALL
    need = oz.ozemu_gated_linear_bytes(4, 4, 8, FAKE + 2, 8, FAKE, 8)
    assert need > 0 and _gated(oz, X=FAKE + 2, nbytes=need - 1) == oz.OZEMU_ERR_SCRATCH_TOO_SMALL
    g, s, t, _ = _arrays(sizes=(1 << 30,))
    need = oz.ozemu_clip_grad_norm_bytes(1, g, s, t)
    assert need > 0 and _clip(oz, sizes=(1 << 30,), nbytes=need - 1) == oz.OZEMU_ERR_SCRATCH_TOO_SMALL
    assert oz.ozemu_clip_grad_norm_bytes(1, *_arrays()[:3]) == 0  # little: one launch, no workspace


def test_queries_on_bad_arguments(oz):
    assert oz.ozemu_gated_linear_bytes(4, 4, 8, FAKE + 2, 7, FAKE, 8) == 0
    assert oz.ozemu_gated_linear_bytes(4, (1 << 25) + 1, 8, FAKE + 2, 8, FAKE, 8) == 0
    assert oz.ozemu_gated_linear_backward_bytes(-1, 4, 8, FAKE, 8, FAKE, 8) == 0
    assert oz.ozemu_clip_grad_norm_bytes(-1, None, None, None) == 0


def test_empty_problems_are_noops(oz):
    assert _gated(oz, m=0, X=NULL, H=NULL, ws=NULL, nbytes=0) == oz.OZEMU_OK
    assert _gated(oz, n=0, W=NULL, H=NULL, bias=NULL, ws=NULL, nbytes=0) == oz.OZEMU_OK
    assert _gated_backward(oz, m=0, n=0, ws=NULL, nbytes=0) == oz.OZEMU_OK
    for empty in (dict(rows=0), dict(k=0)):
        assert _quantize(oz, codes=NULL, scales=NULL, X=NULL, **empty) == oz.OZEMU_OK
        assert _dequantize(oz, codes=NULL, scales=NULL, Y=NULL, **empty) == oz.OZEMU_OK
    assert _mx_linear(oz, m=0, xc=NULL, xs=NULL, Y=NULL) == oz.OZEMU_OK
    assert _mx_linear(oz, n=0, wc=NULL, ws=NULL, Y=NULL, bias=NULL) == oz.OZEMU_OK


def _mx(oz, rows, cols):
    return oz.MXMatrix.empty(rows, cols, device="cpu")


def refused(call):
    with pytest.raises(ValueError) as e:
        call()
    return str(e.value)


def test_binding_refuses_wrong_tensors(oz):
    b16 = torch.bfloat16
    x, w, pre = torch.zeros(2, 4, dtype=b16), torch.zeros(6, 4, dtype=b16), torch.zeros(2, 6, dtype=b16)
    dh = torch.zeros(2, 3, dtype=b16)
    q, wq = _mx(oz, 2, 4), _mx(oz, 3, 4)
    g = torch.zeros(10)
    for bad in (lambda: oz.gated_linear(x, w),                                        # not on the GPU
                lambda: oz.gated_linear(x.float(), w.float()),
                lambda: oz.gated_linear(x, w[:5]),                                    # an odd number of rows
                lambda: oz.gated_linear(x, w.half()), lambda: oz.gated_linear(x, w[:, :3]),
                lambda: oz.gated_linear(x, w, torch.zeros(3, dtype=b16)),
                lambda: oz.gated_linear(x, w, activation="tanh"),
                lambda: oz.gated_linear(x, w, out=torch.zeros(2, 6, dtype=b16)),
                lambda: oz.gated_linear_backward(dh, x, w, None), lambda: oz.gated_linear_backward(dh, x, w, dh),
                lambda: oz.gated_linear_backward(pre, x, w, pre),
                lambda: oz.mx_quantize(x), lambda: oz.mx_quantize(x.double()), lambda: oz.mx_quantize(x[0]),
                lambda: oz.mx_quantize(x.t()), lambda: oz.mx_quantize(x, out=wq), lambda: oz.mx_quantize(x, out=x),
                lambda: oz.mx_dequantize(q), lambda: oz.mx_dequantize(x), lambda: oz.mx_dequantize(q, torch.float64),
                lambda: oz.mx_dequantize(q, out=torch.zeros(2, 5)),
                lambda: oz.mx_dequantize(q, torch.float16, out=torch.zeros(2, 4)),
                lambda: oz.mx_dequantize(oz.MXMatrix(q.data[1:], 2, 4)),
                lambda: oz.mx_dequantize(oz.MXMatrix(q.data.float(), 2, 4)),
                lambda: oz.mx_linear(q, wq), lambda: oz.mx_linear(x, wq), lambda: oz.mx_linear(q, w),
                lambda: oz.mx_linear(q, _mx(oz, 3, 5)), lambda: oz.mx_linear(q, wq, dtype=torch.float32),
                lambda: oz.mx_linear(q, wq, torch.zeros(4, dtype=b16)),
                lambda: oz.mx_linear(q, wq, residual=x), lambda: oz.mx_linear(q, wq, residual=dh, times=dh),
                lambda: oz.mx_linear(q, wq, residual=dh, dtype=torch.float16),
                lambda: oz.mx_linear(oz.MXMatrix(q.data, 200, 4), wq),
                lambda: oz.clip_grad_norm([g], 1.0), lambda: oz.clip_grad_norm([], 1.0),
                lambda: oz.clip_grad_norm([g.double()], 1.0), lambda: oz.clip_grad_norm([g[::2]], 1.0),
                lambda: oz.clip_grad_norm([g[:1].expand(4)], 1.0), lambda: oz.clip_grad_norm([g], 1.0, out=[]),
                lambda: oz.clip_grad_norm([g], 1.0, out=[torch.zeros(9)]),
                lambda: oz.clip_grad_norm([g], 1.0, out=[torch.zeros(10).half()]),
                lambda: oz.clip_grad_norm([torch.zeros(3, 4)], 1.0, out=[torch.zeros(4, 3).t()]),
                lambda: oz.clip_grad_norm([g, 3], 1.0)):
        refused(bad)
    for bad in (lambda: oz.clip_grad_norm(3, 1.0), lambda: oz.clip_grad_norm([g], "one")):
        with pytest.raises(TypeError):
            bad()


def test_outputs_overlap_nothing(oz):
    b16 = torch.bfloat16
    buf = torch.zeros(4096, dtype=b16)

    def view(rows, cols, at, ld=None):
        return torch.as_strided(buf, (rows, cols), (ld or cols, 1), at)
    x, w = view(8, 16, 0), view(12, 16, 200)
    assert "overlaps x" in refused(lambda: oz.gated_linear(x, w, out=view(8, 6, 100)))
    assert "overlaps w" in refused(lambda: oz.gated_linear(x, w, out=view(8, 6, 380)))
    assert "overlaps bias" in refused(lambda: oz.gated_linear(x, w, view(1, 12, 500)[0], out=view(8, 6, 460)))
    assert "CUDA" in refused(lambda: oz.gated_linear(x, w, out=view(8, 6, 128)))
    bytes_ = torch.zeros(20000, dtype=torch.uint8)
    start = -bytes_.data_ptr() % 256

    def mx(rows, cols, at):
        n = _mx(oz, rows, cols).data.numel()
        return oz.MXMatrix(bytes_[start + at:start + at + n], rows, cols)

    def matrix(rows, cols, at):
        return bytes_[start + at:start + at + 2 * rows * cols].view(b16).view(rows, cols)
    q, wq = mx(8, 16, 0), mx(4, 16, 2048)  # 1280 bytes each
    assert "overlaps x" in refused(lambda: oz.mx_quantize(matrix(8, 16, 1024), out=q))
    assert "CUDA" in refused(lambda: oz.mx_quantize(matrix(8, 16, 1280), out=q))
    assert "overlaps q" in refused(lambda: oz.mx_dequantize(q, out=matrix(8, 16, 1264)))
    assert "CUDA" in refused(lambda: oz.mx_dequantize(q, out=matrix(8, 16, 1280)))
    assert "overlaps x" in refused(lambda: oz.mx_linear(q, wq, out=matrix(8, 4, 1264)))
    assert "overlaps w" in refused(lambda: oz.mx_linear(q, wq, out=matrix(8, 4, 3264)))
    r = matrix(8, 4, 1280)
    assert "CUDA" in refused(lambda: oz.mx_linear(q, wq, residual=r, out=r))
    assert "CUDA" in refused(lambda: oz.mx_linear(q, wq, times=r, out=r))
    assert "overlaps residual" in refused(lambda: oz.mx_linear(q, wq, residual=r, out=matrix(8, 4, 1296)))
    assert "overlaps times" in refused(lambda: oz.mx_linear(q, wq, times=r, out=matrix(8, 4, 1296)))
    assert "overlaps bias" in refused(lambda: oz.mx_linear(q, wq, bias=matrix(1, 4, 1280)[0], out=r))
    g = torch.zeros(100)
    parts = [g[:10], g[10:30], g[40:]]
    assert "CUDA" in refused(lambda: oz.clip_grad_norm(parts, 1.0, out=parts))
    assert "CUDA" in refused(lambda: oz.clip_grad_norm([g[:10], g[:10]], 1.0))  # read twice
    assert "another output" in refused(lambda: oz.clip_grad_norm([g[:10], g[:10]], 1.0, out=[g[:10], g[:10]]))
    assert "not its own" in refused(lambda: oz.clip_grad_norm([g[:10], g[10:20]], 1.0, out=[g[10:20], g[:10]]))
    assert "not its own" in refused(lambda: oz.clip_grad_norm([g[:10]], 1.0, out=[g[5:15]]))
    assert "not its own" in refused(lambda: oz.clip_grad_norm([g[:10], g[5:15]], 1.0, out=[g[:10], g[50:60]]))
    assert "not its own" in refused(lambda: oz.clip_grad_norm([g[:40], g[60:70]], 1.0, out=[torch.zeros(40), g[30:40]]))
    assert "CUDA" in refused(lambda: oz.clip_grad_norm([g[:40], g[60:70]], 1.0, out=[torch.zeros(40), g[40:50]]))


# ------------------------------------------------------------------------------------------ launches

WRAPPED = ["cudaLaunchKernelExC", "cudaGetDevice", "cudaFuncSetAttribute", "cudaOccupancyMaxActiveClusters",
           "cudaGetLastError", "cudaGetDriverEntryPointByVersion"]
NO_MEMORY = 2  # cudaErrorMemoryAllocation


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    from ozaki_ii_fp64_gb300 import build
    build.build()
    objects = os.path.join(build.ROOT, "_build", platform.machine())
    exe = str(tmp_path_factory.mktemp("launches") / "feed_forward_launches")
    subprocess.run([build.nvcc()] + build.ARCH_FLAGS + ["-std=c++17", "-I" + build.CSRC,
                   os.path.join(HERE, "feed_forward_launches.cu")]
                   + [os.path.join(objects, name) for name in ("linear.o", "mx.o", "clip.o")] + ["-o", exe]
                   + ["-Xlinker=--wrap=" + name for name in WRAPPED], check=True)

    def run(what, a, b, c=0, odd=0):
        out = subprocess.run([exe, what, str(a), str(b), str(c), str(odd)], check=True, capture_output=True, text=True)
        rows = []
        for line in out.stdout.splitlines():
            status, *grids = line.split()
            rows.append((int(status), [tuple(int(x) for x in g.split(",")) for g in grids]))
        return rows  # without a failure, then with the first launch failing, the second, ...
    return run


@pytest.mark.parametrize("what, a, b, c, odd, count", [
    ("gated", 1000, 4096, 2048, 0, 1), ("gated", 1000, 4096, 2049, 0, 2), ("gated", 3, 4096, 2048, 0, 1),
    ("gated", 5, 9, 0, 0, 1), ("gated_backward", 64, 4096, 4096, 0, 3), ("gated_backward", 1000, 1024, 2048, 0, 3),
    ("gated_backward", 1333, 1025, 2051, 0, 4), ("gated_backward", 100000, 264, 264, 0, 4),
    ("gated_backward", 0, 16, 16, 0, 2), ("quantize", 300, 1000, 0, 1, 1), ("dequantize", 300, 1000, 0, 0, 1),
    ("mx", 1, 4096, 2049, 0, 1), ("mx", 1000, 4096, 2049, 0, 1), ("mx", 5, 9, 0, 0, 1),
    ("clip", 5, 1000, 0, 0, 1), ("clip", 5, 10000000, 0, 0, 2), ("clip", 100, 10, 0, 0, 2), ("clip", 2000, 10, 0, 0, 6)])
def test_each_launch_failure_is_the_calls(launches, what, a, b, c, odd, count):
    (status, grids), *failures = launches(what, a, b, c, odd)
    assert status == 0 and len(grids) == count
    assert len(failures) == count
    for i, (status, tried) in enumerate(failures):
        assert status == NO_MEMORY
        assert tried == grids[:i + 1]  # nothing is launched on what was not made


@pytest.mark.parametrize("what, a, b, c", [
    ("gated", 1 << 26, 9, 16), ("gated", 9, 1 << 25, 16), ("gated", 300, 300, 1 << 26), ("gated", 300, 1 << 25, 16),
    ("gated_backward", 1 << 26, 9, 16), ("gated_backward", 9, 1 << 25, 16), ("gated_backward", 300, 300, 1 << 26),
    ("quantize", 1 << 26, 1, 0), ("quantize", 1, 1 << 26, 0), ("quantize", 1 << 26, 1000, 0), ("dequantize", 1 << 26, 9, 0),
    ("mx", 1 << 26, 9, 16), ("mx", 9, 1 << 26, 16), ("mx", 300, 300, 1 << 26), ("mx", 300, 1 << 26, 16),
    ("clip", 3, 2000000000, 0)])
def test_grids_at_the_size_limits(launches, what, a, b, c):
    # CUDA's limits; a grid that wrapped round is above them.
    (status, grids), *_ = launches(what, a, b, c)
    assert status == 0
    for x, y, z in grids:
        assert 0 < x < 2**31 and 0 < y < 2**16 and 0 < z < 2**16
