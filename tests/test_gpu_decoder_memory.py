"""The examples' captured decoders after everything but the graph and its output has been let go and the memory that could
have been freed is full of other values."""

import gc
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


def load(name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def others(sizes):
    """Tensors of those numbers of bytes, several of each, full of ones."""
    return [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]


def test_gated_decoder():
    example = load("gated_feed_forward")
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(1, 512, generator=gen, device="cuda").to(BF16)
    reference = example.GatedFeedForward(512, 1024, seed=3)
    weights = reference.four_bits()  # of the same seed, made before
    want = reference.decode(x, weights)
    sizes = [w.data.numel() for w in weights] + [2 * 512, 4 * 512, 2 * 512 * 1024, 4 * 512 * 1024]
    graph, y = example.GatedFeedForward(512, 1024, seed=3).decoder(x.clone())
    gc.collect()
    kept = others(sizes)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert all(bool((t == 255).all()) for t in kept)


def test_decoder():
    example = load("feed_forward")
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(1, 512, generator=gen, device="cuda").to(BF16)
    want = example.FeedForward(512, 1024, seed=3).forward(x)[0]
    graph, y = example.FeedForward(512, 1024, seed=3).decoder(x.clone())
    gc.collect()
    kept = others([2 * 512, 4 * 512, 2 * 1024, 2 * 512 * 1024])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert all(bool((t == 255).all()) for t in kept)
