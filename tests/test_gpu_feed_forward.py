"""The feed-forward block of examples/feed_forward.py against the same block in 64 bits with automatic gradients."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def block64(params, x, activation):
    F = torch.nn.functional
    h = F.layer_norm(x, (x.shape[1],), params["norm_weight"], params["norm_bias"])
    z = F.linear(h, params["w1"], params["b1"])
    a = F.gelu(z, approximate="tanh") if activation == "gelu_tanh" else F.silu(z)
    return x + F.linear(a, params["w2"], params["b2"])


# In 2-norm every rounding to 16 bits adds at most its unit roundoff, relative to what is rounded: h, pre, a, y forward;
# da, dz, dh, dx and the saved h, a, pre again backward.  The block's sums of many terms do not amplify a relative
# error of independent roundings; factor 2 for the norm's and the activation's slopes.
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens, hidden, inner, activation", [(1, 256, 512, "silu"), (37, 200, 513, "gelu_tanh"),
                                                               (600, 512, 1024, "gelu_tanh")])
def test_block_forward_and_backward(example, tokens, hidden, inner, activation, dtype):
    block = example.FeedForward(hidden, inner, dtype=dtype, activation=activation, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").to(dtype)
    dy = torch.randn(tokens, hidden, generator=gen, device="cuda").to(dtype)
    y, saved = block.forward(x)
    dx, grads = block.backward(dy, saved)
    params = {k: v.double().requires_grad_() for k, v in block.params.items()}
    xd = x.double().requires_grad_()
    want = block64(params, xd, activation)
    want.backward(dy.double())

    def far(got, ref):
        return float((got.double() - ref).norm() / ref.norm())
    assert far(y, want.detach()) <= 2 * 4 * U[dtype]
    assert far(dx, xd.grad) <= 2 * 8 * U[dtype]
    for name, p in params.items():
        assert far(grads[name], p.grad) <= 2 * 8 * U[dtype], name


def test_decoder_graph_follows_its_input(example):
    block = example.FeedForward(512, 1024, seed=3)
    x = torch.zeros(1, 512, dtype=torch.bfloat16, device="cuda")
    graph, y = block.decoder(x)
    for seed in (4, 5):
        x.copy_(torch.randn(1, 512, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, block.forward(x)[0])


def test_example_runs(example, capsys):
    example.main(256, 512, 1024)
    losses = [float(line.split()[-1]) for line in capsys.readouterr().out.splitlines() if line.startswith("step")]
    assert len(losses) == 4 and all(b < a for a, b in zip(losses, losses[1:]))
