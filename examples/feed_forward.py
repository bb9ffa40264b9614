"""A transformer's feed-forward block on the layer operators: y = x + act(norm(x) W1^T + b1) W2^T + b2.

The block runs a prompt, one training step on it (gradients of every parameter and of x) and a decoded token, the
last as a CUDA graph.

    python examples/feed_forward.py [tokens hidden inner]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ozaki_ii_fp64_gb300 as oz  # noqa: E402


class FeedForward:
    """Parameters in the data's 16-bit type, those of the norm in 32 bits."""

    def __init__(self, hidden, inner, dtype=torch.bfloat16, activation="gelu_tanh", device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (scale * torch.randn(*shape, generator=gen, device=device)).to(dtype)

        self.activation = activation
        self.params = {
            "norm_weight": torch.ones(hidden, device=device), "norm_bias": torch.zeros(hidden, device=device),
            "w1": normal(inner, hidden, scale=hidden ** -0.5), "b1": normal(inner, scale=0.1),
            "w2": normal(hidden, inner, scale=inner ** -0.5), "b2": normal(hidden, scale=0.1),
        }

    def forward(self, x):
        """The block's output, and what its backward pass takes."""
        p = self.params
        h, mean, rstd = oz.layer_norm(x, p["norm_weight"], p["norm_bias"], stats=True)
        a, pre = oz.linear(h, p["w1"], p["b1"], activation=self.activation, save_pre=True)
        y = oz.linear(a, p["w2"], p["b2"], residual=x)
        return y, (x, mean, rstd, h, pre, a)

    def backward(self, dy, saved):
        """dx, and the parameters' gradients."""
        p, (x, mean, rstd, h, pre, a) = self.params, saved
        da, dw2, db2 = oz.linear_backward(dy, a, p["w2"])
        dh, dw1, db1 = oz.linear_backward(da, h, p["w1"], pre, activation=self.activation)
        # The skip connection's gradient joins in the norm's pass.
        dx, dnw, dnb = oz.layer_norm_backward(dh, x, mean, rstd, p["norm_weight"], dresidual=dy)
        return dx, {"norm_weight": dnw, "norm_bias": dnb, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2}

    def decoder(self, x):
        """(graph, output): a replay runs the block on what x holds then, into the output."""
        p = self.params
        hidden, inner = p["w2"].shape
        h, y = torch.empty_like(x), torch.empty_like(x)
        a = torch.empty(x.shape[0], inner, dtype=x.dtype, device=x.device)

        def step():
            oz.layer_norm(x, p["norm_weight"], p["norm_bias"], out=h)
            oz.linear(h, p["w1"], p["b1"], activation=self.activation, out=a)
            oz.linear(a, p["w2"], p["b2"], residual=x, out=y)

        step()  # the first call on a device allocates
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        return graph, y


def timed(f, n=20):
    for _ in range(3):
        f()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(n):
        f()
    end.record()
    torch.cuda.synchronize()
    return begin.elapsed_time(end) / n * 1e3


def main(tokens=4096, hidden=4096, inner=16384):
    block = FeedForward(hidden, inner)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    target = torch.randn(tokens, hidden, device="cuda").bfloat16()
    for step in range(4):  # plain gradient descent on the mean square
        y, saved = block.forward(x)
        error = y.float() - target.float()
        _, grads = block.backward((error * (2 / hidden)).bfloat16(), saved)
        print("step %d: loss %.4f" % (step, float(error.square().mean())))
        for name, p in block.params.items():
            p.sub_((grads[name].float() / tokens).to(p.dtype))
    dy = (error * (2 / hidden)).bfloat16()
    print("forward %.0f us" % timed(lambda: block.forward(x)))
    print("forward and backward %.0f us" % timed(lambda: block.backward(dy, block.forward(x)[1])))
    graph, out = block.decoder(x[:1].clone())
    print("one token %.1f us" % timed(graph.replay))
    if oz.get_status() != oz.OZEMU_OK:
        raise RuntimeError("device status not OK")


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:]))
