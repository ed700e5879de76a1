"""The measured cases of the position-wise layers: layer norm with its backward pass, a dense layer with
bias, activation and residual, and a gated feed-forward projection, each forward and backward.

`run` computes them with the library's calls where `own` is true and in plain torch operations
where it is not; `exact` gives the same results in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid")


def listed():
    return [
        # the norm before a layer while one token is decoded: latency counts
        dict(name="norm one token", op="norm", n=1, d=4096, x="bf16", out="bf16", param="bf16",
             train=False, res=False),
        # a training step's norm of the feature rows of a mini-batch's second frontier: narrow rows whose
        # width is no multiple of a vector, single-precision states, bf16 activations
        dict(name="norm frontier", op="norm", n=180_224, d=100, x="f32", out="bf16", param="f32",
             train=True, res=False),
        # a training step's norm of a batch of long sequences, beside a residual branch
        dict(name="norm tokens", op="norm", n=32_768, d=4096, x="bf16", out="bf16", param="bf16",
             train=True, res=True),
        # the output projection of one token, added to the residual stream
        dict(name="linear one token", op="linear", n=1, d_in=4096, d_out=4096, dtype="bf16",
             act="none", bias=True, res=True, backward=False),
        # odd sizes in every direction, single precision
        dict(name="linear odd", op="linear", n=333, d_in=1030, d_out=2571, dtype="f32", act="gelu",
             bias=True, res=True, backward=False),
        # gradients of the weights [2 d, d_out] of one layer over a mini-batch's first frontier
        dict(name="linear nodes grad", op="linear", n=16_384, d_in=256, d_out=128, dtype="f32",
             act="relu", bias=True, res=False, backward=True),
        # gradients of a feed-forward block's first layer in training
        dict(name="linear tokens grad", op="linear", n=16_384, d_in=1024, d_out=4096, dtype="bf16",
             act="gelu", bias=True, res=False, backward=True),
        # a whole batch's output projection, added to the residual stream
        dict(name="linear large", op="linear", n=16_384, d_in=4096, d_out=4096, dtype="bf16",
             act="none", bias=False, res=True, backward=False),
        # four sequences decode a token each
        dict(name="gated few tokens", op="gated", n=4, d_in=4096, d_out=10_240, dtype="bf16",
             act="silu", bias=False, backward=False),
        # a short ragged batch's gradients, odd sizes, single precision
        dict(name="gated odd grad", op="gated", n=77, d_in=515, d_out=1371, dtype="f32",
             act="gelu_tanh", bias=True, backward=True),
        # a training step's gradients
        dict(name="gated tokens grad", op="gated", n=8192, d_in=2048, d_out=5632, dtype="bf16",
             act="silu", bias=False, backward=True),
        # the forward pass over a whole batch, both projections kept for the backward pass
        dict(name="gated large", op="gated", n=16_384, d_in=4096, d_out=10_240, dtype="bf16",
             act="silu", bias=False, backward=False),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """The same, every other one a multiple of 64 where it is wide enough."""
    d = _spread(rng, lo, hi)
    return d // 64 * 64 if d >= 64 and rng.random() < 0.5 else d


def draw(rng):
    op = rng.choice(["norm", "linear", "gated"])
    if op == "norm":
        d = _width(rng, 16, 16_384)
        return dict(op=op, n=_spread(rng, 1, min(262_144, 134_000_000 // d)), d=d,
                    x=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]),
                    param=rng.choice(["f32", "bf16"]), train=rng.random() < 0.6,
                    res=rng.random() < 0.5)
    dtype, backward = rng.choice(["f32", "bf16"]), rng.random() < 0.5
    # of multiplications and additions, in units of 2 n d_in d_out
    top = 68e9 if dtype == "f32" else 274e9
    top /= (2 if backward else 1) * (2 if op == "gated" else 1)
    while True:
        n = _spread(rng, 1, 32_768)
        d_in, d_out = _width(rng, 16, 10_240), _width(rng, 16, 10_240)
        if n * d_in * d_out <= top:
            break
    case = dict(op=op, n=n, d_in=d_in, d_out=d_out, dtype=dtype, act=rng.choice(ACTIVATIONS),
                bias=rng.random() < 0.5, backward=backward)
    if op == "linear":
        case["res"] = not backward and rng.random() < 0.5
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype, scale=1.0, shift=0.0):
        return (scale * torch.randn(*shape, generator=gen, device="cuda") + shift).to(dtype)

    s = dict(case=case)
    if case["op"] == "norm":
        n, d = case["n"], case["d"]
        x, out, param = DTYPES[case["x"]], DTYPES[case["out"]], DTYPES[case["param"]]
        # a residual stream: columns of their own size and offset
        size = torch.exp(0.5 * torch.randn(d, generator=gen, device="cuda"))
        s["x"] = (size * torch.randn(n, d, generator=gen, device="cuda") +
                  0.5 * torch.randn(d, generator=gen, device="cuda")).to(x)
        s["weight"] = normal(d, dtype=param, scale=0.1, shift=1.0)
        s["bias"] = normal(d, dtype=param, scale=0.1)
        s["out"] = torch.empty(n, d, device="cuda", dtype=out)
        if case["train"]:
            s["mean"], s["rstd"] = (torch.empty(n, device="cuda") for _ in range(2))
            s["dout"] = normal(n, d, dtype=out, scale=1e-2)
            s["dres"] = normal(n, d, dtype=x, scale=1e-2) if case["res"] else None
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"], s["dbias"] = torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
            if own:
                import graph_mini_pipeline_amd as gm
                s["ws"] = torch.empty(gm.gnn_layer_norm_workspace_size(n, d), dtype=torch.uint8,
                                      device="cuda")
        return s
    n, d_in, d_out, dtype = case["n"], case["d_in"], case["d_out"], DTYPES[case["dtype"]]
    gated = case["op"] == "gated"
    s["x"] = normal(n, d_in, dtype=dtype)           # the output of a norm
    names = ("w_gate", "w_up") if gated else ("w",)
    biases = ("bias_gate", "bias_up") if gated else ("bias",)
    kept = ("gate", "up") if gated else ("pre",)
    for w, b in zip(names, biases):
        s[w] = normal(d_in, d_out, dtype=dtype, scale=d_in ** -0.5)
        s[b] = normal(d_out, dtype=dtype, scale=0.1) if case["bias"] else None
    if case["backward"]:
        # what the forward pass kept
        for w, b, z in zip(names, biases, kept):
            s[z] = None
            if gated or case["act"] != "none":
                z32 = s["x"].float() @ s[w].float()
                s[z] = (z32 if s[b] is None else z32 + s[b].float()).to(dtype)
        s["dout"] = normal(n, d_out, dtype=dtype, scale=1e-2)
        for y in ("x",) + names + biases:
            s["d" + y] = None if s[y] is None else torch.empty_like(s[y])
    else:
        s["out"] = torch.empty(n, d_out, device="cuda", dtype=dtype)
        if gated:
            s["gate"], s["up"] = torch.empty_like(s["out"]), torch.empty_like(s["out"])
        else:
            s["res"] = normal(n, d_out, dtype=dtype) if case["res"] else None
            s["pre"] = None if case["act"] == "none" else torch.empty_like(s["out"])
    if own:
        import graph_mini_pipeline_amd as gm
        if gated:
            size = gm.gnn_gated_linear_workspace_size(n, d_in, d_out, dtype, backward=case["backward"])
        else:
            size = gm.gnn_linear_workspace_size(n, d_in, d_out, dtype, backward=case["backward"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def run(s):
    return {"norm": _norm, "linear": _linear, "gated": _gated}[s["case"]["op"]](s)


def _norm(s):
    if own:
        import graph_mini_pipeline_amd as gm
        if not s["case"]["train"]:
            gm.gnn_layer_norm(s["x"], s["weight"], s["bias"], EPS, s["out"])
            return s["out"]
        gm.gnn_layer_norm(s["x"], s["weight"], s["bias"], EPS, s["out"], mean=s["mean"],
                          rstd=s["rstd"])
        gm.gnn_layer_norm_backward(s["x"], s["weight"], s["mean"], s["rstd"], s["dout"], s["dx"],
                                   s["ws"], dweight=s["dweight"], dbias=s["dbias"],
                                   residual_grad=s["dres"])
        return s["out"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"]
    x, w, b = s["x"].float(), s["weight"].float(), s["bias"].float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    x = x * rstd
    out = (x * w + b).to(s["out"].dtype)
    if not s["case"]["train"]:
        return out
    dy = s["dout"].float()
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - x * (g * x).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    dw, db = (dy * x).sum(0), dy.sum(0)
    return (out, mean[:, 0], rstd[:, 0], dx.to(s["x"].dtype), dw.to(s["weight"].dtype),
            db.to(s["bias"].dtype))


def _act(name, z):
    """act(z), act'(z) of a 32-bit z."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        live = z > 0
        return torch.where(live, z, 0.0), live.float()
    if name == "sigmoid":
        y = torch.sigmoid(z)
        return y, y * (1 - y)
    if name == "silu":
        y = torch.sigmoid(z)
        return z * y, y * (1 + z * (1 - y))
    if name == "gelu":
        # the lower tail of the normal distribution, without the difference 1 - erf
        y = 0.5 * torch.erfc(z * -math.sqrt(0.5))
        return z * y, y + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    # gelu_tanh: (1 + tanh t) / 2 = sigmoid(2 t)
    c = 2 * math.sqrt(2 / math.pi)
    y = torch.sigmoid(c * (z + 0.044715 * z * z * z))
    return z * y, y + z * y * (1 - y) * c * (1 + 3 * 0.044715 * z * z)


def _linear(s):
    case = s["case"]
    if own:
        import graph_mini_pipeline_amd as gm
        if not case["backward"]:
            gm.gnn_linear(s["x"], s["w"], s["out"], s["ws"], bias=s["bias"], activation=case["act"],
                          residual=s["res"], pre=s["pre"])
            return s["out"] if s["pre"] is None else (s["out"], s["pre"])
        gm.gnn_linear_backward(s["x"], s["w"], s["dout"], s["ws"], activation=case["act"],
                               pre=s["pre"], dx=s["dx"], dw=s["dw"], dbias=s["dbias"])
        return [s[y] for y in ("dx", "dw", "dbias") if s[y] is not None]
    dtype = s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    if not case["backward"]:
        z = x @ w
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = z if case["act"] == "none" else _act(case["act"], z)[0]
        if s["res"] is not None:
            y = y + s["res"].float()
        return y.to(dtype) if s["pre"] is None else (y.to(dtype), z.to(dtype))
    dz = s["dout"].float()
    if case["act"] != "none":
        dz = dz * _act(case["act"], s["pre"].float())[1]
    grads = [(dz @ w.t()).to(dtype), (x.t() @ dz).to(dtype)]
    if case["bias"]:
        grads.append(dz.sum(0).to(dtype))
    return grads


def _gated(s):
    case = s["case"]
    if own:
        import graph_mini_pipeline_amd as gm
        if not case["backward"]:
            gm.gnn_gated_linear(s["x"], s["w_gate"], s["w_up"], s["out"], s["ws"],
                                bias_gate=s["bias_gate"], bias_up=s["bias_up"],
                                activation=case["act"], gate=s["gate"], up=s["up"])
            return s["out"], s["gate"], s["up"]
        gm.gnn_gated_linear_backward(s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], s["dout"],
                                     s["ws"], activation=case["act"], dx=s["dx"],
                                     dw_gate=s["dw_gate"], dw_up=s["dw_up"],
                                     dbias_gate=s["dbias_gate"], dbias_up=s["dbias_up"])
        return [s[y] for y in ("dx", "dw_gate", "dw_up", "dbias_gate", "dbias_up")
                if s[y] is not None]
    dtype = s["x"].dtype
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    if not case["backward"]:
        g, u = x @ wg, x @ wu
        if case["bias"]:
            g, u = g + s["bias_gate"].float(), u + s["bias_up"].float()
        return (_act(case["act"], g)[0] * u).to(dtype), g.to(dtype), u.to(dtype)
    dy = s["dout"].float()
    a, slope = _act(case["act"], s["gate"].float())
    dg, du = dy * s["up"].float() * slope, dy * a
    grads = [(dg @ wg.t() + du @ wu.t()).to(dtype), (x.t() @ dg).to(dtype), (x.t() @ du).to(dtype)]
    if case["bias"]:
        grads += [dg.sum(0).to(dtype), du.sum(0).to(dtype)]
    return grads


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "norm":
        n, d, zx, zy = case["n"], case["d"], size[case["x"]], size[case["out"]]
        params = 2 * d * size[case["param"]]
        if not case["train"]:
            return dict(bytes=n * d * (zx + zy) + params, flops=8 * n * d)
        # x and dout once, and where there is one the residual branch's gradient
        moved = n * d * ((3 if case["res"] else 2) * zx + 2 * zy)
        return dict(bytes=moved + 8 * n + 2 * params, flops=20 * n * d)
    z, n, d_in, d_out = size[case["dtype"]], case["n"], case["d_in"], case["d_out"]
    mats = 2 if case["op"] == "gated" else 1
    rows_in, rows_out, weights = n * d_in, n * d_out, mats * d_in * d_out
    bias = mats * d_out if case["bias"] else 0
    kept = mats if case["op"] == "gated" or case["act"] != "none" else 0
    flops = 2 * n * weights
    if case["backward"]:
        return dict(bytes=z * (2 * rows_in + (1 + kept) * rows_out + 2 * weights + bias),
                    flops=2 * flops)
    res = 1 if case.get("res") else 0
    return dict(bytes=z * (rows_in + (1 + kept + res) * rows_out + weights + bias), flops=flops)


def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return {"norm": _exact_norm, "linear": _exact_linear, "gated": _exact_gated}[case["op"]](s)


def _exact_norm(s):
    x, w, d = s["x"], s["weight"], s["case"]["d"]
    var, mean = torch.var_mean(x, dim=1, correction=0)
    rstd = (var + EPS) ** -0.5
    scaled = torch.einsum("nd,n->nd", x - mean[:, None], rstd)
    out = torch.addcmul(s["bias"], scaled, w)
    if not s["case"]["train"]:
        return out
    # the gradient of the centred and scaled row, projected off the constant row and off the row itself
    g = s["dout"] * w
    along = torch.linalg.vecdot(g, scaled) / d
    dx = (g - along[:, None] * scaled - g.sum(1)[:, None] / d) * rstd[:, None]
    if s["dres"] is not None:
        dx += s["dres"]
    ones = torch.ones(1, x.shape[0], dtype=torch.float64, device="cuda")
    return out, mean, rstd, dx, (s["dout"] * scaled).sum(0), torch.mm(ones, s["dout"])[0]


def _exact_act(name, z):
    """act(z) in 64 bits, of a z that can be differentiated."""
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return torch.relu(z) if name == "relu" else z


def _slope(name, z):
    z = z.detach().requires_grad_()
    with torch.enable_grad():
        y = _exact_act(name, z)
        return y.detach(), torch.autograd.grad(y.sum(), z)[0]


def _affine(x, w, b):
    return torch.mm(x, w) if b is None else torch.addmm(b, x, w)


def _exact_linear(s):
    case = s["case"]
    if not case["backward"]:
        pre = _affine(s["x"], s["w"], s["bias"])
        y = _exact_act(case["act"], pre)
        if s["res"] is not None:
            y = y + s["res"]
        return y if s["pre"] is None else (y, pre)
    dz = s["dout"]
    if case["act"] != "none":
        dz = dz * _slope(case["act"], s["pre"])[1]
    grads = [torch.mm(dz, s["w"].t()), torch.mm(s["x"].t(), dz)]
    return grads + [dz.sum(0)] if case["bias"] else grads


def _exact_gated(s):
    case = s["case"]
    if not case["backward"]:
        g = _affine(s["x"], s["w_gate"], s["bias_gate"])
        u = _affine(s["x"], s["w_up"], s["bias_up"])
        return _exact_act(case["act"], g) * u, g, u
    y, slope = _slope(case["act"], s["gate"])
    dg, du = s["dout"] * slope * s["up"], s["dout"] * y
    dx = torch.addmm(torch.mm(dg, s["w_gate"].t()), du, s["w_up"].t())
    grads = [dx, torch.mm(s["x"].t(), dg), torch.mm(s["x"].t(), du)]
    return grads + [dg.sum(0), du.sum(0)] if case["bias"] else grads
