"""A transformer's gated feed-forward block: y = x + (act(h Wg^T) * (h Wu^T)) Wd^T with h = norm(x).

The block is trained in 16 bits, its gradients clipped by their global norm, and decodes tokens with its weights in 4 bits
(a CUDA graph).

    python examples/gated_feed_forward.py [tokens hidden inner]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ozaki_ii_fp64_gb300 as oz  # noqa: E402


class GatedFeedForward:
    """Parameters in the data's 16-bit type, those of the norm in 32 bits."""

    def __init__(self, hidden, inner, dtype=torch.bfloat16, activation="silu", device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (scale * torch.randn(*shape, generator=gen, device=device)).to(dtype)

        self.activation, self.inner = activation, inner
        self.params = {
            "norm_weight": torch.ones(hidden, device=device), "norm_bias": torch.zeros(hidden, device=device),
            "w_in": normal(2 * inner, hidden, scale=hidden ** -0.5),  # the gate's rows, then the up projection's
            "w_out": normal(hidden, inner, scale=inner ** -0.5),
        }

    def forward(self, x):
        """The block's output, and what its backward pass takes."""
        p = self.params
        h, mean, rstd = oz.layer_norm(x, p["norm_weight"], p["norm_bias"], stats=True)
        a, pre = oz.gated_linear(h, p["w_in"], activation=self.activation, save_pre=True)
        y = oz.linear(a, p["w_out"], residual=x)
        return y, (x, mean, rstd, h, pre, a)

    def backward(self, dy, saved):
        """dx, and the parameters' gradients."""
        p, (x, mean, rstd, h, pre, a) = self.params, saved
        da, dw_out, _ = oz.linear_backward(dy, a, p["w_out"], bias_grad=False)
        dh, dw_in, _ = oz.gated_linear_backward(da, h, p["w_in"], pre, activation=self.activation, bias_grad=False)
        # The skip connection's gradient joins in the norm's pass.
        dx, dnw, dnb = oz.layer_norm_backward(dh, x, mean, rstd, p["norm_weight"], dresidual=dy)
        return dx, {"norm_weight": dnw, "norm_bias": dnb, "w_in": dw_in, "w_out": dw_out}

    def step(self, grads, rate, max_norm=1.0):
        """Gradient descent with clipped gradients; the norm that they had."""
        held = list(grads.values())
        norm, _ = oz.clip_grad_norm(held, max_norm, out=held)
        for name, p in self.params.items():
            p.sub_((rate * grads[name].float()).to(p.dtype))
        return norm

    def four_bits(self):
        """The block's matrices as 4 bits hold them, for decode."""
        w_in, w_out = self.params["w_in"], self.params["w_out"]
        return oz.mx_quantize(w_in[:self.inner]), oz.mx_quantize(w_in[self.inner:]), oz.mx_quantize(w_out)

    def decode(self, x, weights):
        """The block's output with the products in 4 bits."""
        p, (gate, up, down) = self.params, weights
        h = oz.mx_quantize(oz.layer_norm(x, p["norm_weight"], p["norm_bias"]))
        u = oz.mx_linear(h, up, dtype=x.dtype)
        a = oz.mx_linear(h, gate, activation=self.activation, times=u, out=u)
        return oz.mx_linear(oz.mx_quantize(a), down, residual=x)

    def decoder(self, x):
        """(graph, output): a replay decodes what x holds then, with the block's matrices as they were, into the output."""
        weights = self.four_bits()
        self.decode(x, weights)  # the first call on a device allocates
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.decode(x, weights)
        # A graph keeps no reference to what it reads from outside its own memory.
        graph.reads = x, weights, list(self.params.values())
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


def main(tokens=4096, hidden=4096, inner=8192):
    block = GatedFeedForward(hidden, inner)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    target = torch.randn(tokens, hidden, device="cuda").bfloat16()
    for step in range(4):  # gradient descent on the mean square
        y, saved = block.forward(x)
        error = y.float() - target.float()
        _, grads = block.backward((error * (2 / error.numel())).bfloat16(), saved)
        norm = block.step(grads, 1.0)
        print("step %d: loss %.4f, gradient norm %.4f" % (step, float(error.square().mean()), float(norm)))
    dy = (error * (2 / error.numel())).bfloat16()
    print("forward %.0f us" % timed(lambda: block.forward(x)))
    print("forward and backward %.0f us" % timed(lambda: block.backward(dy, block.forward(x)[1])))
    print("clipping %.0f us" % timed(lambda: oz.clip_grad_norm(list(grads.values()), 1.0, out=list(grads.values()))))
    graph, out = block.decoder(x[:1].clone())
    print("one token with 4-bit weights %.1f us" % timed(graph.replay))
    if oz.get_status() != oz.OZEMU_OK:
        raise RuntimeError("device status not OK")


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:]))
