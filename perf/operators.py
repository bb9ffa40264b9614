"""Cases of the transformer-layer operators: layer norm and the fused linear layer, forward and backward.

`run` takes a state from `prepare` through one operator: in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where `own` is true, through the library's entry points.  `exact` gives the same outputs
from the definitions in 64 bits.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-5

# The largest listed work, which a drawn case keeps within.
MOST_PRODUCTS = 8192 * 4096 * 16384
MOST_ELEMENTS = 16384 * 8192


def listed():
    def norm(name, op, rows, cols, type, wtype, stats=True, residual=False, pad=0):
        return {"name": name, "op": op, "rows": rows, "cols": cols, "type": type, "wtype": wtype, "stats": stats,
                "residual": residual, "pad": pad}

    def lin(name, op, m, k, n, type, act, bias=True, residual=False, save=False, pad=0):
        return {"name": name, "op": op, "m": m, "k": k, "n": n, "type": type, "act": act, "bias": bias,
                "residual": residual, "save": save, "pad": pad}

    return [
        # One decoded token's hidden vector before a layer: pure latency.
        norm("norm_token", "layer_norm", 1, 4096, "bf16", "bf16", stats=False),
        # The hidden states of a training batch, statistics kept for the backward pass.
        norm("norm_batch", "layer_norm", 16384, 8192, "bf16", "bf16"),
        # An odd width in 32 bits, rows taken from a wider matrix.
        norm("norm_odd_f32", "layer_norm", 1021, 5003, "f32", "f32", pad=3),
        # Gradients of the batch, 32-bit parameters, the skip connection's gradient added to dx.
        norm("norm_grad_batch", "layer_norm_backward", 16384, 4096, "bf16", "f32", residual=True),
        # A short ragged batch in 16-bit floats.
        norm("norm_grad_odd_f16", "layer_norm_backward", 777, 2051, "f16", "f16"),
        # The up projection of one decoded token: the weights are read once.
        lin("linear_token", "linear", 1, 4096, 16384, "bf16", "gelu"),
        # The down projection of a few sequences decoded together, added to the residual stream.
        lin("linear_13_tokens_f16", "linear", 13, 16384, 4096, "f16", "none", residual=True),
        # A prompt of no round length through a layer of no round sizes, rows that no 16-byte load fits.
        lin("linear_ragged_f16", "linear", 1000, 2049, 4099, "f16", "silu", residual=True),
        # The up projection of a training batch, the pre-activation kept for the backward pass.
        lin("linear_batch", "linear", 8192, 4096, 16384, "bf16", "gelu_tanh", save=True),
        # A fine-tuning step on few tokens: gradients bound by the weights' bytes.
        lin("linear_grad_tokens_f16", "linear_backward", 64, 4096, 4096, "f16", "none"),
        # Gradients of a ragged layer and batch.
        lin("linear_grad_ragged", "linear_backward", 1333, 2051, 1025, "bf16", "relu"),
        # Gradients of the training batch: two large products.
        lin("linear_grad_batch", "linear_backward", 8192, 4096, 16384, "bf16", "gelu"),
    ]


def draw(rng):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, min(hi, v))

    def width(lo, hi):  # half of the layers have round sizes
        v = size(lo, hi)
        return max(64, v // 64 * 64) if rng.random() < 0.5 else v

    op = rng.choice(("layer_norm", "layer_norm_backward", "linear", "linear_backward"))
    pad = rng.choice((0, 0, 0, 8, 3))
    if op.startswith("layer_norm"):
        type = rng.choice(("bf16", "f16", "f32"))
        while True:
            rows, cols = size(1, 16384), width(32, 16384)
            if rows * cols <= MOST_ELEMENTS:
                break
        return {"op": op, "rows": rows, "cols": cols, "type": type, "wtype": rng.choice((type, "f32")),
                "stats": rng.random() < 0.5, "residual": rng.random() < 0.5, "pad": pad}
    while True:
        m, k, n = size(1, 16384), width(32, 16384), width(32, 16384)
        if m * k * n <= MOST_PRODUCTS:
            break
    return {"op": op, "m": m, "k": k, "n": n, "type": rng.choice(("bf16", "f16")), "act": rng.choice(ACTIVATIONS),
            "bias": rng.random() < 0.75, "residual": rng.random() < 0.5, "save": rng.random() < 0.5, "pad": pad}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = TYPES[case["type"]]

    def normal(rows, cols, scale=1.0, pad=case["pad"], dtype=dt):
        t = torch.randn(rows, cols + pad, generator=gen, device=dev, dtype=torch.float32).mul_(scale).to(dtype)
        return t[:, :cols] if pad else t

    s = dict(case)
    if case["op"].startswith("layer_norm"):
        rows, cols, wt = case["rows"], case["cols"], TYPES[case["wtype"]]
        # Hidden states: an offset, a spread of its own for each row, and a few channels that stand out.
        x = torch.randn(rows, cols + case["pad"], generator=gen, device=dev, dtype=torch.float32)
        x *= torch.rand(rows, 1, generator=gen, device=dev) * 3 + 0.5
        x += 0.25
        x[:, :: max(1, cols // 4)] *= 6
        s["x"] = x.to(dt)[:, :cols]
        s["weight"] = (1 + 0.2 * torch.randn(cols, generator=gen, device=dev)).to(wt)
        s["bias"] = (0.1 * torch.randn(cols, generator=gen, device=dev)).to(wt)
        if case["op"] == "layer_norm_backward":
            s["dy"] = normal(rows, cols)
            s["dresidual"] = normal(rows, cols) if case["residual"] else None
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = (xf - s["mean"][:, None]).square().mean(1).add(EPS).rsqrt()
        return s
    m, k, n = case["m"], case["k"], case["n"]
    s["x"] = normal(m, k)
    s["w"] = normal(n, k, 1 / math.sqrt(k))
    s["b"] = normal(1, n, 0.5, pad=0)[0] if case["bias"] else None
    if case["op"] == "linear":
        s["r"] = normal(m, n) if case["residual"] else None
    else:
        s["dy"] = normal(m, n)
        s["pre"] = normal(m, n) if case["act"] != "none" else None
    return s


# ------------------------------------------------------------------ plain forms

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
    dt, x = s["x"].dtype, s["x"].float()
    if s["op"] == "layer_norm":
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
        y = (d * rstd * s["weight"].float() + s["bias"].float()).to(dt)
        return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]} if s["stats"] else {"y": y}
    if s["op"] == "layer_norm_backward":
        dy = s["dy"].float()
        xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        if s["dresidual"] is not None:
            dx = dx + s["dresidual"].float()
        wt = s["weight"].dtype
        return {"dx": dx.to(dt), "dweight": (dy * xhat).sum(0).to(wt), "dbias": dy.sum(0).to(wt)}
    w = s["w"].float()
    if s["op"] == "linear":
        z = x @ w.t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _activation(z, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return {"y": y.to(dt), "pre": z.to(dt)} if s["save"] else {"y": y.to(dt)}
    dz = s["dy"].float()
    if s["pre"] is not None:
        dz = dz * _slope(s["pre"].float(), s["act"])
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
    if s["op"] == "layer_norm":
        if s["stats"]:
            y, mean, rstd = oz.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, stats=True)
            return {"y": y, "mean": mean, "rstd": rstd}
        return {"y": oz.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)}
    if s["op"] == "layer_norm_backward":
        dx, dweight, dbias = oz.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"],
                                                    dresidual=s["dresidual"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if s["op"] == "linear":
        if s["save"]:
            y, pre = oz.linear(s["x"], s["w"], s["b"], s["r"], activation=s["act"], save_pre=True)
            return {"y": y, "pre": pre}
        return {"y": oz.linear(s["x"], s["w"], s["b"], s["r"], activation=s["act"])}
    dx, dw, db = oz.linear_backward(s["dy"], s["x"], s["w"], s["pre"], activation=s["act"],
                                    bias_grad=s["b"] is not None)
    return {"dx": dx, "dw": dw} if db is None else {"dx": dx, "dw": dw, "db": db}


def run(state):
    return _kernels(state) if own else _plain(state)


def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"].startswith("layer_norm"):
        rows, cols, ws = case["rows"], case["cols"], 4 if case["wtype"] == "f32" else 2
        if case["op"] == "layer_norm":
            return {"bytes": 2 * rows * cols * size + 2 * cols * ws + (8 * rows if case["stats"] else 0),
                    "flops": 8 * rows * cols}
        return {"bytes": (3 + case["residual"]) * rows * cols * size + 3 * cols * ws + 8 * rows,
                "flops": 14 * rows * cols}
    m, k, n = case["m"], case["k"], case["n"]
    if case["op"] == "linear":
        outs = 1 + case["residual"] + case["save"]
        return {"bytes": size * (m * k + n * k + outs * m * n + case["bias"] * n), "flops": 2 * m * n * k}
    pre = case["act"] != "none"
    return {"bytes": size * (2 * m * k + 2 * n * k + (1 + pre) * m * n + case["bias"] * n), "flops": 4 * m * n * k}


# --------------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    F = torch.nn.functional
    phi = {"none": lambda z: z, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
           "gelu_tanh": lambda z: F.gelu(z, approximate="tanh")}
    x = s["x"].double()
    if case["op"] == "layer_norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        y = F.layer_norm(x, (case["cols"],), s["weight"].double(), s["bias"].double(), EPS)
        return {"y": y, "mean": mean, "rstd": (var + EPS) ** -0.5} if case["stats"] else {"y": y}
    if case["op"] == "layer_norm_backward":
        # d/dx of sum(dy * (xhat w + b)) with xhat = (x - mean) rstd and both statistics functions of x:
        # the projection of the scaled gradient off the constant and xhat directions.
        dy, rstd = s["dy"].double(), s["rstd"].double().unsqueeze(1)
        xhat = torch.sub(x, s["mean"].double().unsqueeze(1)).mul_(rstd)
        g = torch.einsum("ij,j->ij", dy, s["weight"].double())
        along = torch.einsum("ij,ij->i", g, xhat).div_(case["cols"])
        dx = g.sub(g.sum(1, keepdim=True) / case["cols"]).sub_(xhat * along.unsqueeze(1)).mul_(rstd)
        if s["dresidual"] is not None:
            dx += s["dresidual"]
        return {"dx": dx, "dweight": torch.einsum("ij,ij->j", dy, xhat), "dbias": torch.einsum("ij->j", dy)}
    if case["op"] == "linear":
        z = F.linear(x, s["w"].double(), None if s["b"] is None else s["b"].double())
        y = phi[case["act"]](z)
        if s["r"] is not None:
            y = y + s["r"]
        return {"y": y, "pre": z} if case["save"] else {"y": y}
    dz = s["dy"].double()
    if s["pre"] is not None:
        z = s["pre"].double().requires_grad_()
        dz, = torch.autograd.grad(phi[case["act"]](z), z, dz)
    r = {"dx": torch.einsum("ij,jk->ik", dz, s["w"].double()), "dw": torch.einsum("ij,ik->jk", dz, x)}
    if s["b"] is not None:
        r["db"] = torch.einsum("ij->j", dz)
    return r
