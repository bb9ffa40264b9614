"""The gated block of examples/gated_feed_forward.py: its training step against the same block in 64 bits with automatic
gradients, its decoding against the products of the 4-bit values in 64 bits."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# In 2-norm every rounding to 16 bits adds at most its unit roundoff, relative to what is rounded; a sum of many terms
# does not amplify a relative error of independent roundings.  Factor 2 for the slopes of the norm and the activation.
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(ROOT, "examples", "gated_feed_forward.py")
    spec = importlib.util.spec_from_file_location("gated_feed_forward", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def far(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens, hidden, inner, activation", [(1, 256, 512, "silu"), (37, 200, 513, "gelu_tanh"),
                                                               (600, 512, 1024, "gelu")])
def test_training_step(example, tokens, hidden, inner, activation, dtype):
    F = torch.nn.functional
    block = example.GatedFeedForward(hidden, inner, dtype=dtype, activation=activation, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").to(dtype)
    dy = torch.randn(tokens, hidden, generator=gen, device="cuda").to(dtype)
    params = {k: v.double().requires_grad_() for k, v in block.params.items()}
    xd = x.double().requires_grad_()
    h = F.layer_norm(xd, (hidden,), params["norm_weight"], params["norm_bias"])
    gate, up = F.linear(h, params["w_in"]).chunk(2, 1)
    act = {"silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda z: F.gelu(z, approximate="tanh")}[activation]
    want = xd + F.linear(act(gate) * up, params["w_out"])
    want.backward(dy.double())
    y, saved = block.forward(x)
    dx, grads = block.backward(dy, saved)
    # Roundings forward: h (twice, through gate and up), a, y; backward: da, both halves of dz, dh, dx, and the saved ones.
    assert far(y, want.detach()) <= 2 * 5 * U[dtype]
    assert far(dx, xd.grad) <= 2 * 10 * U[dtype]
    for name, p in params.items():
        assert far(grads[name], p.grad) <= 2 * 10 * U[dtype], name
    norm64 = float(sum(p.grad.square().sum() for p in params.values())) ** 0.5
    before = {k: v.clone() for k, v in block.params.items()}
    norm = float(block.step(grads, 0.5, max_norm=0.25))
    assert abs(norm - norm64) <= 2 * 10 * U[dtype] * norm64
    for name, p in params.items():  # the gradients themselves are clipped, and the step is theirs
        assert far(grads[name], p.grad * min(1.0, 0.25 / (norm64 + 1e-6))) <= 2 * 21 * U[dtype], name
        assert torch.equal(block.params[name], before[name] - (0.5 * grads[name].float()).to(before[name].dtype)), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens, hidden, inner", [(1, 512, 1024), (9, 200, 513), (700, 256, 2048)])
def test_decoding(example, tokens, hidden, inner, dtype):
    oz = example.oz
    F = torch.nn.functional
    block = example.GatedFeedForward(hidden, inner, dtype=dtype, seed=3)
    x = torch.randn(tokens, hidden, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(dtype)
    weights = block.four_bits()
    gate, up, down = (oz.mx_dequantize(w, torch.float32).double() for w in weights)
    # Each step from the same 16-bit values as the block's own: a value next to a border may take either code.
    h = oz.mx_quantize(oz.layer_norm(x, block.params["norm_weight"], block.params["norm_bias"]))
    hd = oz.mx_dequantize(h, torch.float32).double()
    u = oz.mx_linear(h, weights[1], dtype=dtype)
    assert far(u, F.linear(hd, up)) <= 2 * U[dtype]
    a = oz.mx_linear(h, weights[0], activation="silu", times=u)
    assert far(a, F.silu(F.linear(hd, gate)) * u.double()) <= 2 * U[dtype]
    ad = oz.mx_dequantize(oz.mx_quantize(a), torch.float32).double()
    y = block.decode(x, weights)
    assert far(y, x.double() + F.linear(ad, down)) <= 2 * U[dtype]


def test_decoder_graph_follows_its_input(example):
    block = example.GatedFeedForward(512, 1024, seed=3)
    x = torch.zeros(1, 512, dtype=torch.bfloat16, device="cuda")
    graph, y = block.decoder(x)
    weights = block.four_bits()
    for seed in (4, 5):
        x.copy_(torch.randn(1, 512, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, block.decode(x, weights))


def test_example_runs(example, capsys):
    example.main(256, 512, 1024)
    assert sum(line.startswith("step") for line in capsys.readouterr().out.splitlines()) == 4
