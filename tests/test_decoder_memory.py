"""What a captured decoder of the examples reads and writes lives as long as its graph: a CUDA graph itself keeps no reference
to memory from outside its capture.  On the host, with a stand-in for the capture and plain operators."""

import contextlib
import gc
import importlib.util
import os
import types
import weakref

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Graph:
    def replay(self):
        pass


class Held:
    """Stands for an MXMatrix: its data is what a replay reads."""

    def __init__(self, w):
        self.data = w.clone()


def load(name, oz, monkeypatch):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.oz = oz
    monkeypatch.setattr(torch.cuda, "CUDAGraph", Graph)
    monkeypatch.setattr(torch.cuda, "graph", lambda graph: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "synchronize", lambda: None)
    return module


def check(read, make):
    """The tensors that the captured calls took (in `read`) are there after everything but the graph is gone."""
    graph = make()
    gc.collect()
    assert read and all(ref() is not None for ref in read)
    del graph
    gc.collect()
    assert not any(ref() is not None for ref in read)  # and no longer than the graph


def test_gated_decoder(monkeypatch):
    read = []

    def see(*tensors):
        read[:] = read[-20:] + [weakref.ref(t) for t in tensors if t is not None]

    def norm(x, w, b):
        see(x, w, b)
        return x + 0

    def quantize(x):
        return Held(x)

    def linear(x, w, residual=None, activation="none", dtype=None, times=None, out=None):
        see(w.data, residual)
        return x.data @ w.data.t()

    oz = types.SimpleNamespace(layer_norm=norm, mx_quantize=quantize, mx_linear=linear)
    example = load("gated_feed_forward", oz, monkeypatch)

    def make():
        block = example.GatedFeedForward(8, 12, device="cpu")
        graph, y = block.decoder(torch.zeros(1, 8, dtype=torch.bfloat16))
        read[:] = read[-7:]  # of the captured step: x, the norm's parameters, three weights, the residual
        return graph
    check(read, make)


def test_decoder(monkeypatch):
    read = []

    def norm(x, w, b, out):
        read.extend(weakref.ref(t) for t in (x, w, b, out))

    def linear(x, w, b, out, activation="none", residual=None):
        read.extend(weakref.ref(t) for t in (x, w, b, out) + ((residual,) if residual is not None else ()))

    example = load("feed_forward", types.SimpleNamespace(layer_norm=norm, linear=linear), monkeypatch)

    def make():
        block = example.FeedForward(8, 12, device="cpu")
        graph, y = block.decoder(torch.zeros(1, 8, dtype=torch.bfloat16))
        return graph
    check(read, make)
