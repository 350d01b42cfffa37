"""64-bit restatements of the group norm and 8-bit product operators (numpy, straight from
their definitions) and the tolerances the GPU tests hold the kernels to.

Tolerances, from the roundings a kernel makes (u = 2^-24 for FP32, 2^-9 for one BF16 rounding):
  * group norm, FP32: h = (x - mean) * rstd carries the rounding of the mean (u * |mean| * rstd),
    of rstd (a sum of n values in a tree of short chains: < 64 u) and three products; gamma,
    beta and the activation add a few u of their own terms.  1e-5 = 168 u of (1 + |y|) plus
    8 u |mean| rstd |gamma| covers them.
  * a BF16 result: one rounding, 2^-8 |y| leaves it a factor of two, on top of the FP32 bound.
  * backward: the same 1e-5 of the sum of the magnitudes of dx's three terms; dgamma and dbeta
    1e-5 of the sum of the magnitudes they add up.
  * 8-bit product: the integer sum is exact below 2^24, then four roundings and the activation:
    16 u of (|sum * scales| + |bias|), plus 2^-8 |y| for BF16.  Past 2^24 each of the K / 16
    accumulations may lose 2^-23 of the magnitudes added so far.
"""
import numpy as np

U32 = 2.0 ** -24
F32_TOL = 1e-5
BF16_TOL = 2.0 ** -8


def activation(z, act):
    if act == "relu":
        return np.where(np.isnan(z), z, np.maximum(z, 0.0))
    if act == "silu":
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-z))
    return z


def activation_grad(z, act):
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "silu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def per_channel(stat, C):
    """[N][G] -> [N][1][C]"""
    return np.repeat(stat, C // stat.shape[1], axis=1)[:, None, :]


def norm_stats(x, groups, eps):
    """mean and rstd [N][G] of x [N][P][C]."""
    N, P, C = x.shape
    v = x.reshape(N, P, groups, C // groups)
    mean = v.mean(axis=(1, 3))
    var = ((v - mean[:, None, :, None]) ** 2).mean(axis=(1, 3))
    return mean, 1.0 / np.sqrt(var + eps)


def norm_forward(x, groups, gamma, beta, eps, act):
    """y, and the FP32 tolerance of each of its values."""
    C = x.shape[2]
    mean, rstd = norm_stats(x, groups, eps)
    m, r = per_channel(mean, C), per_channel(rstd, C)
    z = (x - m) * r * gamma + beta
    y = activation(z, act)
    return y, F32_TOL * (1.0 + np.abs(z)) + 8 * U32 * np.abs(m * r * gamma)


def norm_backward(dy, x, stats, groups, gamma, beta, act):
    """(dx, dgamma, dbeta) and their FP32 tolerances, from FP32 stats [2][N][G].  ReLU's kink is
    taken where FP32 arithmetic in the operator's order of operations puts it."""
    N, P, C = x.shape
    m, r = per_channel(stats[0].astype(np.float64), C), per_channel(stats[1].astype(np.float64), C)
    h = (x - m) * r
    z = h * gamma + beta
    if act == "relu":
        f = np.float32
        z32 = (x.astype(f) - m.astype(f)) * r.astype(f) * gamma.astype(f) + beta.astype(f)
        grad = (z32 > 0).astype(np.float64)
    else:
        grad = activation_grad(z, act)
    u = dy * grad
    dbeta, dgamma = u.sum((0, 1)), (u * h).sum((0, 1))
    d = u * gamma

    def group_mean(v):
        return per_channel(v.reshape(N, P, groups, C // groups).mean(axis=(1, 3)), C)

    a, b = group_mean(d), group_mean(d * h)
    dx = r * (d - a - h * b)
    big = np.abs(dy) * (1.0 + np.abs(z)) if act == "silu" else np.abs(u)
    group_big = group_mean(big * np.abs(gamma)), group_mean(big * np.abs(gamma) * np.abs(h))
    tol = F32_TOL * r * (big * np.abs(gamma) + group_big[0] + np.abs(h) * group_big[1])
    return (dx, dgamma, dbeta), (tol, F32_TOL * (big * np.abs(h)).sum((0, 1)), F32_TOL * big.sum((0, 1)))


def quantize_rows(x32):
    """q and scale of FP32 rows [M][K]: every operation rounded once in FP32."""
    f = np.float32
    amax = np.max(np.abs(x32), axis=1)
    bad = ~np.isfinite(amax)
    zero = ~bad & (amax < f(2.0 ** -100))
    use = np.where(bad | zero, f(1), amax).astype(f)
    inv, scale = f(127) / use, use / f(127)
    with np.errstate(invalid="ignore"):
        q = np.rint((x32 * inv[:, None]).astype(f))
    q = np.where((bad | zero)[:, None], 0, q).astype(np.int8)
    return q, np.where(bad, f("nan"), np.where(zero, f(0), scale)).astype(f)


def int8_product(xq, xs, wq, ws, bias, act):
    """y [M][N] and the FP32 tolerance of each of its values."""
    a, b = xq.astype(np.float64), wq.astype(np.float64)
    total, size = a @ b.T, np.abs(a) @ np.abs(b).T  # exact: below 2^53
    scales = xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
    bias = np.zeros(len(ws)) if bias is None else bias.astype(np.float64)
    z = total * scales + bias
    lost = np.where(size < 2.0 ** 24, 0.0, np.ceil(xq.shape[1] / 16) * 2.0 ** -23 * size)
    tol = 16 * U32 * (np.abs(total * scales) + np.abs(bias)) + np.abs(scales) * lost
    return activation(z, act), tol


def check(got, ref, tol, bf16, what=""):
    """Every value of `got` within `tol` of `ref`, with one BF16 rounding on top where it has one."""
    assert got.shape == ref.shape, (got.shape, ref.shape)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), what + ": NaN in other places"
    err = np.abs(got - ref)[~nan]
    bound = (tol + (BF16_TOL * np.abs(ref) if bf16 else 0.0))[~nan]
    worst = float(np.max(err - bound)) if err.size else 0.0
    assert worst <= 0.0, "%s: %.3e above its tolerance (largest error %.3e)" % (what, worst, float(err.max()))
