"""Cases of the 16-bit linear layer, the root-mean-square norm and dropout: what is timed and compared.

The residual branch of a layer, in training and in serving: the matrix product of BF16 rows
(tokens, pixels) and weights with bias, activation and residual in its epilogue, and its
gradients; the root-mean-square norm of rows with the residual's addition, its gradients, and
its form that writes 8-bit rows with a scale each for the 8-bit product; dropout whose mask comes
from a counter-based generator (Philox 4x32 of ten rounds) and is never stored.

`own` false: the operators in plain torch, 32 bits throughout, rounded once at the end.
`own` true: the package's functional entry points.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
MAX_LINEAR_FLOPS = 2.8e11          # the largest listed product
MAX_LINEAR_BYTES = 530_000_000     # the pointwise layer with its residual
MAX_ROWS_BYTES = 270_000_000       # the largest listed norm: read x and the residual, write both
MAX_DROPOUT_VALUES = 8192 * 4096


# ---------------------------------------------------------------- cases
def _linear(name, op, M, K, N, act, bias=True, residual=False, z=False):
    c = {"op": op, "M": M, "K": K, "N": N, "act": act}
    if op == "linear":
        c.update(bias=bias, residual=residual, z=z)
    return dict(c, name=name) if name else c


def _rows(name, op, M, C, dtype, residual=True, **more):
    c = {"op": op, "M": M, "C": C, "dtype": dtype, "residual": residual}
    c.update(more)
    return dict(c, name=name) if name else c


def listed():
    return [
        # serving: a single token through a square layer, added to the residual stream
        _linear("linear one token", "linear", 1, 4096, 4096, "none", bias=False, residual=True),
        # ragged in every direction: a short prompt, odd widths
        _linear("linear ragged", "linear", 301, 1000, 777, "silu", residual=True),
        # the block's pointwise layer over a batch of maps, with a skip connection
        _linear("linear pointwise layer", "linear", 200704, 256, 512, "relu", residual=True),
        # a batch of tokens in training: the values before the activation are kept for the gradient
        _linear("linear many tokens", "linear", 8192, 4096, 4096, "silu", z=True),
        # training at odd sizes
        _linear("linear backward ragged", "linear backward", 301, 1000, 777, "relu"),
        # training, the widening half of a layer
        _linear("linear backward many tokens", "linear backward", 8192, 1024, 4096, "silu"),
        # few rows of an odd width, FP32: all latency
        _rows("norm few rows f32", "norm", 5, 1003, "f32"),
        # a batch of tokens: addition to the residual stream, norm
        _rows("norm many tokens", "norm", 8192, 4096, "bf16"),
        # its gradients, with the one that comes down the residual stream
        _rows("norm backward", "norm backward", 8192, 4096, "bf16"),
        # addition, norm, 8-bit rows, product of 8-bit integers
        _rows("norm and 8-bit product", "norm product", 4096, 1024, "bf16", N=4096),
        # a small odd tensor in FP32
        _rows("dropout ragged f32", "dropout", 301, 777, "f32", p=0.1),
        # a batch of tokens, dropped and added to the residual stream
        _rows("dropout many tokens", "dropout", 8192, 4096, "bf16", p=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.4 else max(lo, n // 64 * 64) if n >= 128 else (n + 7) // 8 * 8


def draw(rng):
    while True:
        op = rng.choice(["linear", "linear", "linear", "linear backward", "linear backward", "norm", "norm backward",
                         "norm product", "dropout"])
        M = _log_int(rng, 1, 65536)
        if op.startswith("linear"):
            c = _linear(None, op, M, _width(rng, 32, 8192), _width(rng, 32, 8192), rng.choice(["none", "relu", "silu"]),
                        bias=rng.random() < 0.5, residual=rng.random() < 0.5, z=rng.random() < 0.25)
            w = work(c)
            if w["flops"] <= MAX_LINEAR_FLOPS and w["bytes"] <= MAX_LINEAR_BYTES:
                return c
            continue
        c = _rows(None, op, M, _width(rng, 32, 16384), "bf16" if op == "norm product" else rng.choice(["bf16", "f32"]),
                  residual=rng.random() < 0.7)
        if op == "dropout":
            c["p"] = rng.choice([0.05, 0.1, 0.25, 0.5])
            if c["M"] * c["C"] <= MAX_DROPOUT_VALUES:
                return c
            continue
        if op == "norm product":
            c["N"] = _width(rng, 32, 4096)
        w = work(c)
        if w["bytes"] <= MAX_ROWS_BYTES and w["flops"] <= MAX_LINEAR_FLOPS:
            return c


def work(case):
    c = case
    M = c["M"]
    if c["op"] == "linear":
        K, N = c["K"], c["N"]
        b = 2 * (M * K + N * K + M * N * (1 + c["residual"] + c["z"])) + 4 * N * c["bias"]
        return {"bytes": b, "flops": 2 * M * K * N}
    if c["op"] == "linear backward":
        K, N = c["K"], c["N"]
        z = 0 if c["act"] == "none" else M * N
        return {"bytes": 2 * (M * N + z + 2 * M * K + 2 * N * K) + 4 * N, "flops": 4 * M * K * N}
    C, e = c["C"], 2 if c["dtype"] == "bf16" else 4
    r = 1 if c["residual"] else 0
    if c["op"] == "norm":
        return {"bytes": M * C * e * (2 + 2 * r) + 4 * C, "flops": 5 * M * C}
    if c["op"] == "norm backward":
        return {"bytes": M * C * e * (3 + r) + 8 * C + 4 * M, "flops": 10 * M * C}
    if c["op"] == "dropout":
        return {"bytes": M * C * e * (2 + r) + 16, "flops": 2 * M * C}
    N = c["N"]
    return {"bytes": M * C * e * (1 + 2 * r) + 4 * C + N * C + 8 * N + 2 * M * N, "flops": 2 * M * C * N + 5 * M * C}


# ---------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _rows_of(g, M, C, dtype):
    """Rows as they leave a layer: channels of their own spread, rows of their own size."""
    x = _randn(g, M, C)
    x.mul_(torch.rand(C, device="cuda", generator=g) + 0.5).mul_(torch.rand((M, 1), device="cuda", generator=g) + 0.5)
    return x.to(TORCH[dtype])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    M = c["M"]
    if c["op"].startswith("linear"):
        K, N = c["K"], c["N"]
        c["x"] = _rows_of(g, M, K, "bf16")
        c["w"] = _randn(g, N, K).mul_(1.0 / math.sqrt(K)).to(torch.bfloat16)
        b = _randn(g, N).mul_(0.3)
        if c["op"] == "linear":
            c["b"] = b if c["bias"] else None
            c["r"] = _rows_of(g, M, N, "bf16") if c["residual"] else None
        else:
            c["dy"] = _randn(g, M, N).to(torch.bfloat16)
            # what the forward pass keeps: the values before the activation, in BF16
            c["zs"] = None if c["act"] == "none" else (c["x"] @ c["w"].t()).add_(b.to(torch.bfloat16))
        return c
    C = c["C"]
    c["x"] = _rows_of(g, M, C, c["dtype"])
    if c["op"] == "dropout":
        c["r"] = _rows_of(g, M, C, c["dtype"]) if c["residual"] else None
        c["state"] = torch.randint(0, 1 << 62, (2,), device="cuda", generator=g)  # seed and offset
        return c
    c["gamma"] = _randn(g, C) * 0.2 + 1.0
    c["r"] = _rows_of(g, M, C, c["dtype"]) if c["residual"] else None
    if c["op"] == "norm backward":
        c["dy"] = _randn(g, M, C).to(TORCH[c["dtype"]])
        c["rstd"] = (c["x"].float().square_().mean(1) + EPS).rsqrt()  # what the forward pass leaves
    if c["op"] == "norm product":
        N = c["N"]
        c["w"] = _randn(g, N, C).mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
        c["ws"] = (torch.rand(N, device="cuda", generator=g) + 0.5) / (36.0 * math.sqrt(C))
    return c


# ---------------------------------------------------------------- plain forms
def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"]
    y = z.clamp_min(0.0) if s["act"] == "relu" else z / (1.0 + torch.exp(-z)) if s["act"] == "silu" else z
    if s["r"] is not None:
        y = y + s["r"].float()
    y = y.to(torch.bfloat16)
    return (y, z.to(torch.bfloat16)) if s["z"] else y


def _plain_linear_backward(s):
    x, w, u = s["x"].float(), s["w"].float(), s["dy"].float()
    if s["act"] == "relu":
        u = u * (s["zs"] > 0)
    elif s["act"] == "silu":
        z = s["zs"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        u = u * (sig * (1.0 + z * (1.0 - sig)))
    return (u @ w).to(torch.bfloat16), (u.t() @ x).to(torch.bfloat16), u.sum(0)


def _plain_norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    rstd = (h.square().mean(1, keepdim=True) + EPS).rsqrt()
    return h * rstd * s["gamma"], h.to(s["x"].dtype)


def _plain_norm_backward(s):
    h, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    n = h * rstd
    d = dy * s["gamma"]
    dx = rstd * (d - n * (d * n).mean(1, keepdim=True))
    if s["r"] is not None:
        dx = dx + s["r"].float()
    return dx.to(s["x"].dtype), (dy * n).sum(0)


def _plain_norm_product(s):
    """8-bit rows: scale = amax / 127, q = round(y * (127 / amax)) (rows are finite and not zero here)."""
    y, h = _plain_norm(s)
    amax = y.abs().amax(1, keepdim=True)
    top = torch.full_like(amax, 127.0)  # tensor by tensor: torch divides by a number through its reciprocal
    q = torch.round(y * (top / amax))
    out = ((q @ s["w"].float().t()) * (amax / top) * s["ws"]).to(torch.bfloat16)
    return (out, h) if s["r"] is not None else out


def _times(x, m):
    """The high and low halves of x * m, both below 2^32, in 64-bit integers with a sign."""
    low = x * (m & 0xFFFF)
    mid = x * (m >> 16) + (low >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)


def _plain_words(state, n):
    """The generator's first n 32-bit words for a state (seed, offset): word i % 4 of the block whose
    counter is (i / 4, offset) and whose key is the seed."""
    i = torch.arange((n + 3) // 4, device=state.device)
    mask = 0xFFFFFFFF
    key0, key1 = state[0] & mask, (state[0] >> 32) & mask
    a, b = i & mask, i >> 32
    c, d = (state[1] & mask).expand_as(i), ((state[1] >> 32) & mask).expand_as(i)
    for _ in range(10):
        hi0, lo0 = _times(a, 0xD2511F53)
        hi1, lo1 = _times(c, 0xCD9E8D57)
        a, b, c, d = hi1 ^ b ^ key0, lo1, hi0 ^ d ^ key1, lo0
        key0, key1 = (key0 + 0x9E3779B9) & mask, (key1 + 0xBB67AE85) & mask
    return torch.stack((a, b, c, d), 1).view(-1)[:n]


def _plain_dropout(s):
    x = s["x"].float()
    keep = _plain_words(s["state"], x.numel()).view(x.shape) >= round(s["p"] * 2 ** 32)
    y = torch.where(keep, x * (1.0 / (1.0 - s["p"])), torch.zeros_like(x))
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(s["x"].dtype)


def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "linear":
        return _plain_linear(s)
    if s["op"] == "linear backward":
        return _plain_linear_backward(s)
    if s["op"] == "norm":
        y, h = _plain_norm(s)
        y = y.to(s["x"].dtype)
        return (y, h) if s["r"] is not None else y
    if s["op"] == "norm backward":
        return _plain_norm_backward(s)
    if s["op"] == "norm product":
        return _plain_norm_product(s)
    return _plain_dropout(s)


def _run_own(s):
    import cnn_convolution_implicit_gb300 as cg
    if s["op"] == "linear":
        if s["z"]:
            z = torch.empty((s["M"], s["N"]), dtype=torch.bfloat16, device="cuda")
            return cg.linear(s["x"], s["w"], s["b"], act=s["act"], residual=s["r"], z=z), z
        return cg.linear(s["x"], s["w"], s["b"], act=s["act"], residual=s["r"])
    if s["op"] == "linear backward":
        return cg.linear_backward(s["dy"], s["x"], s["w"], z=s["zs"], act=s["act"])
    if s["op"] == "norm":
        return cg.rms_norm(s["x"], s["gamma"], residual=s["r"], eps=EPS)
    if s["op"] == "norm backward":
        return cg.rms_norm_backward(s["dy"], s["x"], s["rstd"], s["gamma"], dh=s["r"])
    if s["op"] == "norm product":
        q, scale, *h = cg.rms_norm_int8(s["x"], s["gamma"], residual=s["r"], eps=EPS)
        y = cg.int8_matmul(q, scale, s["w"], s["ws"])
        return (y, h[0]) if h else y
    return cg.dropout(s["x"], s["p"], s["state"], residual=s["r"])


# ---------------------------------------------------------------- 64 bits, from the definitions
def _philox(seed, offset, n):
    """The published generator in unsigned 64-bit arithmetic on the host."""
    u = np.uint64
    w32, mask = u(32), u(0xFFFFFFFF)
    i = np.arange((n + 3) // 4, dtype=np.uint64)
    x = [i & mask, i >> w32, np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p, q = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(q >> w32) ^ x[1] ^ u(k0), q & mask, (p >> w32) ^ x[3] ^ u(k1), p & mask]
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    return np.stack(x, 1).reshape(-1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if s["op"] == "linear":
        z = torch.einsum("mk,nk->mn", d["x"], d["w"])
        if "b" in d:
            z += d["b"]
        y = torch.where(z > 0, z, torch.zeros_like(z)) if s["act"] == "relu" else z * torch.sigmoid(z) if s["act"] == "silu" else z
        if "r" in d:
            y = y + d["r"]
        return (y, z) if s["z"] else y
    if s["op"] == "linear backward":
        u = d["dy"]
        if s["act"] == "relu":
            u = torch.where(d["zs"] > 0, u, torch.zeros_like(u))
        elif s["act"] == "silu":
            sg = torch.sigmoid(d["zs"])
            u = u * (sg + d["zs"] * sg * (1.0 - sg))
        return torch.einsum("mn,nk->mk", u, d["w"]), torch.einsum("mn,mk->nk", u, d["x"]), u.sum(0)
    if s["op"] == "dropout":
        seed_, offset = (int(v) for v in s["state"])
        kept = _philox(seed_, offset, d["x"].numel()).astype(np.int64)
        kept = (torch.from_numpy(kept).to("cuda") / 2.0 ** 32 >= round(s["p"] * 2 ** 32) / 2.0 ** 32).view(d["x"].shape)
        y = d["x"] * kept / (1.0 - s["p"])
        return y + d["r"] if "r" in d else y
    if s["op"] == "norm backward":
        M, C = d["x"].shape
        a = d["rstd"].view(M, 1)
        up = d["dy"] * d["gamma"]
        dot = torch.einsum("mc,mc->m", up, d["x"]).view(M, 1)
        dx = a * up - d["x"] * (a ** 3 * dot / C)
        if "r" in d:
            dx += d["r"]
        return dx, torch.einsum("mc,mc->c", d["dy"], d["x"] * a)
    h = d["x"] + d["r"] if "r" in d else d["x"]
    y = h / torch.sqrt(torch.einsum("mc,mc->m", h, h) / h.shape[1] + EPS)[:, None] * d["gamma"]
    if s["op"] == "norm":
        return (y, h) if "r" in d else y
    top = y.abs().max(dim=1).values
    q = torch.round(127.0 * y / top[:, None])
    out = torch.einsum("mc,nc->mn", q, s["w"].double()) * torch.outer(top / 127.0, d["ws"])
    return (out, h) if "r" in d else out
