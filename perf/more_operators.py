"""Cases of the feed-forward operators beyond the plain layer: 4-bit microscaled matrices and their product, the gated
linear layer forward and backward, and clipping gradients by their global norm.

`run` takes a state from `prepare` through one operator: in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where `own` is true, through the library's entry points.  `exact` gives the same outputs
from the definitions in 64 bits.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-6

# The largest listed work, which a drawn case keeps within.
MOST_PRODUCTS = 8192 * 4096 * 16384
MOST_ELEMENTS = 16384 * 8192
MOST_GRADIENTS = 8 * 2 * 4096 * 16384


def listed():
    def quant(name, rows, cols, type, pad=0):
        return {"name": name, "op": "mx_quantize", "rows": rows, "cols": cols, "type": type, "pad": pad}

    def mx(name, m, k, n, type, act, bias=True, residual=False, pad=0):
        return {"name": name, "op": "mx_linear", "m": m, "k": k, "n": n, "type": type, "act": act, "bias": bias,
                "residual": residual, "pad": pad}

    def gated(name, op, m, k, n, type, act, bias=False, save=False, pad=0):
        return {"name": name, "op": op, "m": m, "k": k, "n": n, "type": type, "act": act, "bias": bias, "save": save,
                "pad": pad}

    def clip(name, layers, hidden, inner, type, flat=False, limit=1.0):
        return {"name": name, "op": "clip_grad_norm", "layers": layers, "hidden": hidden, "inner": inner, "type": type,
                "flat": flat, "limit": limit}

    return [
        # The weights of a layer, brought to 4 bits and read back.
        quant("quantize_weights", 16384, 8192, "bf16"),
        # A ragged batch of hidden states in 32 bits, rows taken from a wider matrix.
        quant("quantize_odd_f32", 1021, 5003, "f32", pad=3),
        # One decoded token through a layer of 4-bit weights: the weights are read once.
        mx("mx_linear_token", 1, 4096, 16384, "bf16", "gelu"),
        # A prompt of no round length through a layer of no round sizes.
        mx("mx_linear_ragged_f16", 1000, 2049, 4099, "f16", "silu", residual=True),
        # A long prompt, or a batch of them, through the layer.
        mx("mx_linear_batch", 8192, 4096, 16384, "bf16", "gelu_tanh"),
        # One decoded token through the gated half of a feed-forward block.
        gated("gated_token", "gated_linear", 1, 4096, 8192, "bf16", "silu"),
        # The same for a training batch, both pre-activations kept for the backward pass.
        gated("gated_batch", "gated_linear", 8192, 4096, 8192, "bf16", "silu", save=True),
        # Gradients of a ragged layer and batch.
        gated("gated_grad_ragged_f16", "gated_linear_backward", 1333, 2051, 1025, "f16", "gelu_tanh", bias=True),
        # Gradients of the training batch: a pass over the gradients, and two large products.
        gated("gated_grad_batch", "gated_linear_backward", 8192, 4096, 8192, "bf16", "silu"),
        # The gradients of one small block: latency.
        clip("clip_small", 1, 256, 1024, "bf16"),
        # Gradients of three layers of no round sizes, packed into one buffer without gaps.
        clip("clip_odd_f32", 3, 1021, 4099, "f32", flat=True),
        # The gradients of eight large blocks.
        clip("clip_model", 8, 4096, 16384, "bf16"),
    ]


def draw(rng):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, min(hi, v))

    def width(lo, hi):  # half of the layers have round sizes
        v = size(lo, hi)
        return max(64, v // 64 * 64) if rng.random() < 0.5 else v

    op = rng.choice(("mx_quantize", "mx_linear", "gated_linear", "gated_linear_backward", "clip_grad_norm"))
    pad = rng.choice((0, 0, 0, 8, 3))
    if op == "mx_quantize":
        while True:
            rows, cols = size(1, 16384), width(32, 16384)
            if rows * cols <= MOST_ELEMENTS:
                break
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(("bf16", "f16", "f32")), "pad": pad}
    if op == "clip_grad_norm":
        while True:
            layers, hidden, inner = rng.randint(1, 10), width(32, 4096), width(32, 16384)
            if layers * 2 * hidden * inner <= MOST_GRADIENTS:
                break
        return {"op": op, "layers": layers, "hidden": hidden, "inner": inner, "type": rng.choice(("bf16", "f16", "f32")),
                "flat": rng.random() < 0.5, "limit": rng.choice((1.0, 1.0, 1e6))}
    halves = 1 if op == "mx_linear" else 2
    while True:
        m, k, n = size(1, 16384), width(32, 16384), width(32, 16384)
        if m * k * n * halves <= MOST_PRODUCTS:
            break
    c = {"op": op, "m": m, "k": k, "n": n, "type": rng.choice(("bf16", "f16")), "act": rng.choice(ACTIVATIONS),
         "bias": rng.random() < 0.5, "pad": pad}
    if op == "mx_linear":
        c["residual"] = rng.random() < 0.5
    else:
        c["save"] = rng.random() < 0.5
    return c


def _spread(rows, cols, gen, dev):
    """Hidden states or weights: a spread of its own for each row, and a few channels that stand out."""
    x = torch.randn(rows, cols, generator=gen, device=dev, dtype=torch.float32)
    x *= torch.rand(rows, 1, generator=gen, device=dev) * 3 + 0.5
    x[:, :: max(1, cols // 4)] *= 6
    return x


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = TYPES[case["type"]]
    s = dict(case)
    if case["op"] == "clip_grad_norm":
        # Of each layer: the matrices and biases in its type, the norm's parameters in 32 bits.
        h, i = case["hidden"], case["inner"]
        shapes = [(h,), (h,), (i, h), (i,), (h, i), (h,)] * case["layers"]
        kinds = [torch.float32, torch.float32, dt, dt, dt, dt] * case["layers"]
        counts = [math.prod(x) for x in shapes]
        scale = 4 / math.sqrt(sum(counts))  # a norm of about 4

        def buffers(fill):
            if not case["flat"]:
                return [fill(c, t).view(x) for c, t, x in zip(counts, kinds, shapes)]
            at, whole = {}, {t: fill(sum(c for c, u in zip(counts, kinds) if u == t), t) for t in set(kinds)}
            views = []
            for c, t, x in zip(counts, kinds, shapes):
                views.append(whole[t][at.get(t, 0):at.get(t, 0) + c].view(x))
                at[t] = at.get(t, 0) + c
            return views

        s["grads"] = buffers(lambda c, t: torch.zeros(c, device=dev, dtype=t))
        for g in s["grads"]:
            g.copy_(torch.randn(g.shape, generator=gen, device=dev).mul_(scale * (0.5 + torch.rand(
                (), generator=gen, device=dev))))
        s["out"] = buffers(lambda c, t: torch.empty(c, device=dev, dtype=t))
        return s

    def normal(rows, cols, scale=1.0, pad=case["pad"]):
        t = torch.randn(rows, cols + pad, generator=gen, device=dev, dtype=torch.float32).mul_(scale).to(dt)
        return t[:, :cols] if pad else t

    if case["op"] == "mx_quantize":
        s["x"] = _spread(case["rows"], case["cols"] + case["pad"], gen, dev).to(dt)[:, :case["cols"]]
        return s
    m, k, n = case["m"], case["k"], case["n"]
    if case["op"] == "mx_linear":
        s["x"] = _spread(m, k + case["pad"], gen, dev).to(dt)[:, :k]
        # The layer's weights as 4 bits hold them, kept by either side in its own form.
        s["w"] = _values(_spread(n, k, gen, dev).mul_(1 / math.sqrt(k))).to(dt)
        s["wq"] = _oz().mx_quantize(s["w"]) if own else None
        s["b"] = normal(1, n, 0.5, pad=0)[0] if case["bias"] else None
        s["r"] = normal(m, n) if case["residual"] else None
        return s
    s["x"] = normal(m, k)
    s["w"] = normal(2 * n, k, 1 / math.sqrt(k))
    s["b"] = normal(1, 2 * n, 0.5, pad=0)[0] if case["bias"] else None
    if case["op"] == "gated_linear_backward":
        s["dh"] = normal(m, n)
        s["pre"] = normal(m, 2 * n)
    return s


# ------------------------------------------------------------------ plain forms

def _values(x):
    """The values that 4 bits hold of the rows of x: in each 32 columns a scale 2^(e - 2), e the exponent of the largest
    magnitude, and 0, 0.5, 1, 1.5, 2, 3, 4 or 6 of it, the nearest (the even code between two), 6 beyond."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -cols % 32)).view(rows, -1, 32)
    exponent = torch.frexp(x.abs().amax(2, keepdim=True))[1] - 1
    a = torch.ldexp(x.abs(), 2 - exponent)
    v = 0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75)
    v = v + 1.0 * (a > 2.5) + 1.0 * (a >= 3.5) + 2.0 * (a > 5.0)
    return (torch.ldexp(v, exponent - 2) * torch.sign(x)).view(rows, -1)[:, :cols]


def _activation(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _plain(s):
    if s["op"] == "clip_grad_norm":
        norm = torch.sqrt(torch.stack([(g.float() * g.float()).sum() for g in s["grads"]]).sum())
        factor = (s["limit"] / (norm + EPS)).clamp(max=1.0)
        return {"norm": norm, "clipped": [(g.float() * factor).to(g.dtype) for g in s["grads"]]}
    dt = s["x"].dtype
    if s["op"] == "mx_quantize":
        return {"y": _values(s["x"]).to(dt)}
    x, w, n = s["x"].float(), s["w"].float(), s["n"]
    if s["op"] == "mx_linear":
        z = _values(x) @ w.t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _activation(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return {"y": y.to(dt)}
    if s["op"] == "gated_linear":
        z = x @ w.t()
        if s["b"] is not None:
            z = z + s["b"].float()
        h = _activation(z[:, :n], s["act"]) * z[:, n:]
        return {"h": h.to(dt), "pre": z.to(dt)} if s["save"] else {"h": h.to(dt)}
    dh, g, u = s["dh"].float(), s["pre"][:, :n].float(), s["pre"][:, n:].float()
    dz = torch.cat((dh * u * _slope(g, s["act"]), dh * _activation(g, s["act"])), 1)
    r = {"dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt)}
    if s["b"] is not None:
        r["db"] = dz.sum(0).to(dt)
    return r


# ------------------------------------------------------- the library's operators

_library = None


def _oz():
    global _library
    if _library is None:
        import ozaki_ii_fp64_gb300
        _library = ozaki_ii_fp64_gb300
    return _library


def _kernels(s):
    oz = _oz()
    if s["op"] == "clip_grad_norm":
        norm, clipped = oz.clip_grad_norm(s["grads"], s["limit"], eps=EPS, out=s["out"])
        return {"norm": norm, "clipped": clipped}
    if s["op"] == "mx_quantize":
        return {"y": oz.mx_dequantize(oz.mx_quantize(s["x"]), s["x"].dtype)}
    if s["op"] == "mx_linear":
        return {"y": oz.mx_linear(oz.mx_quantize(s["x"]), s["wq"], s["b"], s["r"], activation=s["act"],
                                  dtype=s["x"].dtype)}
    if s["op"] == "gated_linear":
        if s["save"]:
            h, pre = oz.gated_linear(s["x"], s["w"], s["b"], activation=s["act"], save_pre=True)
            return {"h": h, "pre": pre}
        return {"h": oz.gated_linear(s["x"], s["w"], s["b"], activation=s["act"])}
    dx, dw, db = oz.gated_linear_backward(s["dh"], s["x"], s["w"], s["pre"], activation=s["act"],
                                          bias_grad=s["b"] is not None)
    return {"dx": dx, "dw": dw} if db is None else {"dx": dx, "dw": dw, "db": db}


def run(state):
    return _kernels(state) if own else _plain(state)


def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "clip_grad_norm":
        h, i, layers = case["hidden"], case["inner"], case["layers"]
        count = layers * (2 * h * i + h + i)
        return {"bytes": 2 * (count * size + layers * 2 * h * 4), "flops": 3 * count}
    if case["op"] == "mx_quantize":
        return {"bytes": 2 * case["rows"] * case["cols"] * size, "flops": 4 * case["rows"] * case["cols"]}
    m, k, n = case["m"], case["k"], case["n"]
    if case["op"] == "mx_linear":  # weights of 4 bits, and a byte for 32 of them
        return {"bytes": size * (m * k + (1 + case["residual"]) * m * n + case["bias"] * n) + n * k * 17 // 32,
                "flops": 2 * m * n * k}
    if case["op"] == "gated_linear":
        return {"bytes": size * (m * k + 2 * n * k + (1 + 2 * case["save"]) * m * n + case["bias"] * 2 * n),
                "flops": 4 * m * n * k}
    return {"bytes": size * (2 * m * k + 4 * n * k + 3 * m * n + case["bias"] * 2 * n), "flops": 8 * m * n * k}


# --------------------------------------------------------- definitions in 64 bits

def _held(x):
    """The values of 4 bits and a power of two, by rounding to a grid of 1/2, 1 or 2 steps (half to even)."""
    rows, cols = x.shape
    blocks = -(-cols // 32)
    t = torch.zeros(rows, blocks * 32, dtype=torch.float64, device=x.device)
    t[:, :cols] = x
    t = t.view(rows, blocks, 32)
    most = t.abs().max(2, keepdim=True).values
    scale = torch.exp2(torch.floor(torch.log2(most.clamp(min=2.0 ** -126))) - 2)
    # log2 of a value next to a power of two may round across it.
    scale = torch.where(most >= 8 * scale, 2 * scale, torch.where(most < 4 * scale, scale / 2, scale))
    t = t / scale
    step = torch.where(t.abs() >= 4, 2.0, torch.where(t.abs() >= 2, 1.0, 0.5)).to(t.dtype)
    t = (torch.round(t / step) * step).clamp(-6, 6) * scale
    return t.view(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    F = torch.nn.functional
    phi = {"none": lambda z: z, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
           "gelu_tanh": lambda z: F.gelu(z, approximate="tanh")}
    if case["op"] == "clip_grad_norm":
        norm = torch.stack([torch.linalg.vector_norm(g.double()) for g in s["grads"]]).norm()
        factor = min(1.0, case["limit"] / (float(norm) + EPS))
        return {"norm": norm, "clipped": [g.double() * factor for g in s["grads"]]}
    if case["op"] == "mx_quantize":
        return {"y": _held(s["x"].double())}
    n, w = case["n"], s["w"].double()
    if case["op"] == "mx_linear":
        y = phi[case["act"]](F.linear(_held(s["x"].double()), w, None if s["b"] is None else s["b"].double()))
        return {"y": y if s["r"] is None else y + s["r"]}
    x = s["x"].double()
    if case["op"] == "gated_linear":
        z = F.linear(x, w, None if s["b"] is None else s["b"].double())
        gate, up = z.chunk(2, 1)
        h = phi[case["act"]](gate).mul_(up)
        return {"h": h, "pre": z} if case["save"] else {"h": h}
    z = s["pre"].double().requires_grad_()
    gate, up = z.split(n, 1)
    dz, = torch.autograd.grad(phi[case["act"]](gate) * up, z, s["dh"].double())
    r = {"dx": torch.einsum("ij,jk->ik", dz, w), "dw": torch.einsum("ij,ik->jk", dz, x)}
    if s["b"] is not None:
        r["db"] = torch.einsum("ij->j", dz)
    return r
