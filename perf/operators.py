"""Cases of the normalisation and 8-bit product operators: what is timed and compared.

group norm with an activation over NHWC tensors (forward, backward, and the form that
writes 8-bit integers with one scale per pixel) and the product of 8-bit integers with a
scale for each row (token, pixel) and each output channel.

`own` false: the operators in plain torch, 32 bits throughout, rounded once at the end.
`own` true: the package's functional entry points.
"""
import math

import torch

own = False

EPS = 1e-5
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
MAX_NORM_BYTES = 410_000_000       # the largest listed group norm: read x, write y
MAX_PRODUCT_FLOPS = 2.7e11         # the largest listed product
MAX_PRODUCT_BYTES = 300_000_000


# ---------------------------------------------------------------- cases
def _norm(name, op, N, H, W, C, groups, dtype, act, **more):
    c = {"op": op, "N": N, "H": H, "W": W, "C": C, "groups": groups, "dtype": dtype, "act": act}
    c.update(more)
    return dict(c, name=name) if name else c


def _product(name, M, K, N, x, out, act):
    c = {"op": "product", "M": M, "K": K, "N": N, "x": x, "out": out, "act": act}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one small feature map at the bottom of an image network: all latency
        _norm("norm one 8x8 map", "norm", 1, 8, 8, 256, 32, "bf16", "silu"),
        # ragged FP32 map, 15 channels to a group
        _norm("norm ragged f32", "norm", 5, 61, 47, 120, 8, "f32", "silu"),
        # behind the 112x112 body convolution, its whole batch
        _norm("norm body layer", "norm", 32, 112, 112, 256, 32, "bf16", "relu"),
        # training, behind the FP32 3x3 layer
        _norm("norm backward f32", "backward", 8, 56, 56, 64, 16, "f32", "relu"),
        # training, behind the 64x64 dilated layer
        _norm("norm backward", "backward", 16, 64, 64, 256, 32, "bf16", "silu"),
        # training, the body layer's input
        _norm("norm backward body layer", "backward", 32, 112, 112, 128, 32, "bf16", "relu"),
        # serving: a single token through a square layer
        _product("product one token", 1, 4096, 4096, "bf16", "bf16", "none"),
        # ragged in every direction, rows that start at odd multiples of 8 bytes
        _product("product ragged", 301, 1000, 777, "int8", "f32", "none"),
        # the block's pointwise layer from its BF16 activations, scaled row by row in the call
        _product("product pointwise layer", 200704, 256, 512, "bf16", "bf16", "relu"),
        # a batch of tokens, inputs that are 8-bit already
        _product("product many tokens", 8192, 4096, 4096, "int8", "bf16", "none"),
        # norm, activation, 8-bit pixels, pointwise product: a small map
        _norm("norm and product small", "norm product", 2, 16, 16, 128, 16, "bf16", "silu", C_out=384),
        # the same at the pointwise layer's size
        _norm("norm and product layer", "norm product", 64, 56, 56, 256, 32, "bf16", "silu", C_out=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "backward", "product", "product", "norm product"])
        if op == "product":
            c = _product(None, _log_int(rng, 1, 65536), _log_int(rng, 32, 4096), _log_int(rng, 16, 4096),
                         rng.choice(["bf16", "int8"]), rng.choice(["bf16", "f32"]), rng.choice(["none", "relu", "silu"]))
        else:
            groups = rng.choice([1, 2, 4, 8, 16, 32])
            C = groups * _log_int(rng, 1, 64)
            c = _norm(None, op, _log_int(rng, 1, 32), _log_int(rng, 4, 128), _log_int(rng, 4, 128), C, groups,
                      "bf16" if op == "norm product" else rng.choice(["bf16", "f32"]),
                      rng.choice(["none", "relu", "silu"]))
            if C > 1024 or C < 16:
                continue
            if op == "norm product":
                c["C_out"] = _log_int(rng, 16, 1024)
        w = work(c)
        if w["flops"] <= MAX_PRODUCT_FLOPS and w["bytes"] <= (MAX_PRODUCT_BYTES if "product" in op else MAX_NORM_BYTES):
            return c


def work(case):
    c = case
    if c["op"] == "product":
        M, K, N = c["M"], c["K"], c["N"]
        x = M * K * 2 if c["x"] == "bf16" else M * K + M * 4
        return {"bytes": x + N * K + N * 8 + M * N * (2 if c["out"] == "bf16" else 4), "flops": 2 * M * K * N}
    e = 2 if c["dtype"] == "bf16" else 4
    pixels, C = c["N"] * c["H"] * c["W"], c["C"]
    if c["op"] == "norm":
        return {"bytes": 2 * pixels * C * e + C * 8, "flops": 8 * pixels * C}
    if c["op"] == "backward":
        return {"bytes": 3 * pixels * C * e + C * 16 + c["N"] * c["groups"] * 8, "flops": 20 * pixels * C}
    Co = c["C_out"]
    return {"bytes": pixels * C * e + C * 8 + Co * C + Co * 8 + pixels * Co * 2, "flops": 2 * pixels * C * Co + 8 * pixels * C}


# ---------------------------------------------------------------- inputs
def _map(g, c):
    """A feature map as a convolution leaves it: each channel with its own mean and spread."""
    N, H, W, C = c["N"], c["H"], c["W"], c["C"]
    x = torch.randn((N, H, W, C), device="cuda", generator=g)
    x.mul_(torch.rand(C, device="cuda", generator=g) * 1.5 + 0.25)
    x.add_(torch.randn(C, device="cuda", generator=g) * 0.7)
    return x.to(TORCH[c["dtype"]])


def _weights8(g, N, K):
    """8-bit weights with one scale per output channel, as a quantiser of Gaussian weights leaves them."""
    w = torch.randn((N, K), device="cuda", generator=g).mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
    scale = (torch.rand(N, device="cuda", generator=g) + 0.5) / (36.0 * math.sqrt(K))
    return w, scale, torch.randn(N, device="cuda", generator=g) * 0.1


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if c["op"] == "product":
        M, K, N = c["M"], c["K"], c["N"]
        if c["x"] == "int8":
            c["xq"] = torch.randn((M, K), device="cuda", generator=g).mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
            c["xs"] = (torch.rand(M, device="cuda", generator=g) + 0.5) / 36.0
        else:
            c["xb"] = torch.randn((M, K), device="cuda", generator=g).to(torch.bfloat16)
        c["w"], c["ws"], c["bias"] = _weights8(g, N, K)
        return c
    c["x_map"] = _map(g, c)
    c["gamma"] = torch.randn(c["C"], device="cuda", generator=g) * 0.2 + 1.0
    c["beta"] = torch.randn(c["C"], device="cuda", generator=g) * 0.2
    if c["op"] == "backward":
        c["dy"] = torch.randn(c["x_map"].shape, device="cuda", generator=g).to(TORCH[c["dtype"]])
        v = c["x_map"].float().view(c["N"], -1, c["groups"], c["C"] // c["groups"])
        mean = v.mean((1, 3))
        var = (v - mean[:, None, :, None]).square_().mean((1, 3))
        c["stats"] = torch.stack((mean, (var + EPS).rsqrt()))  # what the forward pass leaves: [2][N][groups]
    if c["op"] == "norm product":
        c["w"], c["ws"], c["bias"] = _weights8(g, c["C_out"], c["C"])
    return c


# ---------------------------------------------------------------- plain forms
def _act(z, act):
    return z.clamp_min(0.0) if act == "relu" else z / (1.0 + torch.exp(-z)) if act == "silu" else z


def _plain_norm(s):
    x = s["x_map"].float()
    v = x.view(s["N"], -1, s["groups"], s["C"] // s["groups"])
    mean = v.mean((1, 3), keepdim=True)
    t = v - mean
    rstd = (t.square().mean((1, 3), keepdim=True) + EPS).rsqrt()
    return _act((t * rstd).view(x.shape) * s["gamma"] + s["beta"], s["act"])


def _plain_backward(s):
    shape = (s["N"], s["H"] * s["W"], s["groups"], s["C"] // s["groups"])
    x, dy = s["x_map"].float().view(shape), s["dy"].float().view(shape)
    mean, rstd = (t.view(s["N"], 1, s["groups"], 1) for t in s["stats"])
    gamma, beta = s["gamma"].view(shape[2:]), s["beta"].view(shape[2:])
    xhat = (x - mean) * rstd
    z = xhat * gamma + beta
    if s["act"] == "relu":
        dy = dy * (z > 0)
    elif s["act"] == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        dy = dy * (sig * (1.0 + z * (1.0 - sig)))
    dgamma, dbeta = (dy * xhat).sum((0, 1)).view(-1), dy.sum((0, 1)).view(-1)
    d = dy * gamma
    dx = rstd * (d - d.mean((1, 3), keepdim=True) - xhat * (d * xhat).mean((1, 3), keepdim=True))
    return dx.view(s["x_map"].shape).to(s["x_map"].dtype), dgamma, dbeta


def _plain_rows8(x):
    """8-bit rows: scale = amax / 127, q = round(x * (127 / amax)) (rows are finite and not zero here)."""
    amax = x.abs().amax(1, keepdim=True)
    top = torch.full_like(amax, 127.0)  # tensor by tensor: torch divides by a number through its reciprocal
    return torch.round(x * (top / amax)), (amax / top).view(-1)


def _plain_product(xq, xs, s, act, out):
    y = (xq.float() @ s["w"].float().t()) * xs[:, None] * s["ws"] + s["bias"]
    return _act(y, act).to(TORCH[out])


def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "norm":
        return _plain_norm(s).to(s["x_map"].dtype)
    if s["op"] == "backward":
        return _plain_backward(s)
    if s["op"] == "product":
        xq, xs = (s["xq"], s["xs"]) if s["x"] == "int8" else _plain_rows8(s["xb"].float())
        return _plain_product(xq, xs, s, s["act"], s["out"])
    xq, xs = _plain_rows8(_plain_norm(s).view(-1, s["C"]))
    return _plain_product(xq, xs, s, "none", "bf16").view(s["N"], s["H"], s["W"], -1)


def _run_own(s):
    import cnn_convolution_implicit_gb300 as cg
    if s["op"] == "norm":
        return cg.group_norm(s["x_map"], s["groups"], s["gamma"], s["beta"], eps=EPS, act=s["act"])
    if s["op"] == "backward":
        return cg.group_norm_backward(s["dy"], s["x_map"], s["stats"], s["groups"], s["gamma"], s["beta"], eps=EPS,
                                      act=s["act"])
    if s["op"] == "product":
        if s["x"] == "int8":
            return cg.int8_matmul(s["xq"], s["xs"], s["w"], s["ws"], s["bias"], act=s["act"], out=s["out"])
        return cg.int8_linear(s["xb"], s["w"], s["ws"], s["bias"], act=s["act"], out=s["out"])
    q, scale = cg.group_norm_int8(s["x_map"], s["groups"], s["gamma"], s["beta"], eps=EPS, act=s["act"])
    return cg.int8_matmul(q, scale, s["w"], s["ws"], s["bias"], act="none", out="bf16")


# ---------------------------------------------------------------- 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)

    def activation(z):
        if s["act"] == "relu":
            return torch.where(z > 0, z, torch.zeros_like(z))
        return z * torch.sigmoid(z) if s["act"] == "silu" else z

    def product(xq, xs):
        out = (xq.double() @ s["w"].double().T) * torch.outer(xs.double(), s["ws"].double()) + s["bias"].double()
        return out

    def rows(x):
        top = x.abs().max(dim=1).values
        return torch.round(127.0 * x / top[:, None]), top / 127.0

    if s["op"] == "product":
        xq, xs = (s["xq"], s["xs"]) if s["x"] == "int8" else rows(s["xb"].double())
        return activation(product(xq, xs))
    N, G, C = s["N"], s["groups"], s["C"]
    x = s["x_map"].double().reshape(N, -1, C)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dgamma, dbeta = (torch.zeros(C, dtype=torch.float64, device="cuda") for _ in range(2))
    gamma, beta = s["gamma"].double(), s["beta"].double()
    for n in range(N):  # one image at a time
        v = x[n].reshape(-1, G, C // G).transpose(0, 1).reshape(G, -1)
        if s["op"] == "backward":  # the statistics are inputs
            mu, r = s["stats"][0, n].double(), s["stats"][1, n].double()
        else:
            var, mu = torch.var_mean(v, dim=1, correction=0)
            r = 1.0 / torch.sqrt(var + EPS)
        h = (x[n] - mu.repeat_interleave(C // G)) * r.repeat_interleave(C // G)
        z = h * gamma + beta
        if s["op"] != "backward":
            y[n] = activation(z)
            continue
        up = s["dy"][n].double().reshape(-1, C)
        if s["act"] == "relu":
            up = torch.where(z > 0, up, torch.zeros_like(up))
        elif s["act"] == "silu":
            sg = torch.sigmoid(z)
            up = up * (sg + z * sg * (1.0 - sg))
        dgamma += (up * h).sum(0)
        dbeta += up.sum(0)
        d = up * gamma
        per_group = d.shape[0] * (C // G)
        a = (d.sum(0).reshape(G, -1).sum(1) / per_group).repeat_interleave(C // G)
        b = ((d * h).sum(0).reshape(G, -1).sum(1) / per_group).repeat_interleave(C // G)
        dx[n] = (d - a - h * b) * r.repeat_interleave(C // G)
    if s["op"] == "norm":
        return y.reshape(s["x_map"].shape)
    if s["op"] == "backward":
        return dx.reshape(s["x_map"].shape), dgamma, dbeta
    q, scale = rows(y.reshape(-1, C))
    return product(q, scale).reshape(N, s["H"], s["W"], -1)
