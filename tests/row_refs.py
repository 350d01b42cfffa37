"""64-bit restatements of the linear layer, the root-mean-square norm and dropout (numpy, straight from
their definitions) and the tolerances the GPU tests hold the kernels to; check() is operator_refs'.

Tolerances, from the roundings a kernel makes (u = 2^-24; a BF16 result adds its rounding in check()):
  * norm: h = x + residual is rounded once, the sum of squares adds positive terms in chains of up to 128
    and a tree (< 150 u of it, halved by the root), then three products: 1e-5 = 168 u of |y|, plus the
    smallest normal numbers' spacing.  Backward: 1e-5 of the sum of the magnitudes of dx's terms; dgamma
    1e-5 of the magnitudes it adds up.
  * linear: products of two BF16 values are exact in FP32.  A tensor core may lose 2^-23 of the
    magnitudes added so far with every 16 products; the joins of parts and the bias add 8 more.  SiLU is
    off by (|z| + 3) u of its value and steeper than 1 by less than 1.1, ReLU not at all.
  * its gradients: u = dy act'(z) is off by 16 (1 + |z|) u of |dy| and, where there is an activation, rounded to
    BF16 (half a step, 2^-8) for dx and dw; dbias adds it unrounded, in chains and a tree: 1e-5 of the magnitudes.
  * dropout: the factor, the product and the sum are rounded: 4 u of |x| / (1 - p) + |residual|.
"""
import numpy as np

from operator_refs import F32_TOL, U32, activation, activation_grad

TINY = 2.0 ** -126
BF16_HALF_STEP = 2.0 ** -8


def rms_forward(x, gamma, r, eps):
    """(y, tolerance), (h, tolerance), rstd"""
    h = x + r if r is not None else x
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None] * gamma
    return (y, F32_TOL * np.abs(y) + TINY), (h, U32 * np.abs(h) + TINY), rstd


def rms_backward(dy, h, rstd, gamma, dh):
    n, d = h * rstd[:, None], dy * gamma
    dot = (d * n).mean(1, keepdims=True)
    size = rstd[:, None] * (np.abs(d) + np.abs(n) * np.abs(d * n).mean(1, keepdims=True))
    dx = rstd[:, None] * (d - n * dot)
    if dh is not None:
        dx, size = dx + dh, size + np.abs(dh)
    return (dx, F32_TOL * size + TINY), ((dy * n).sum(0), F32_TOL * np.abs(dy * n).sum(0) + TINY)


def linear(x, w, bias, r, act):
    """(y, tolerance), (z, tolerance)"""
    z, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        z, size = z + bias, size + np.abs(bias)
    tol = (np.ceil(x.shape[1] / 16) + 8) * 2.0 ** -23 * size
    y = activation(z, act)
    ytol = 1.1 * tol + (np.abs(z) + 8) * U32 * np.abs(y)
    if r is not None:
        ytol = ytol + 2 * U32 * np.abs(r)
        y = y + r
    return (y, ytol + TINY), (z, tol + TINY)


def linear_backward(dy, x, w, z, act):
    """(dx, tolerance), (dw, tolerance), (dbias, tolerance)"""
    u = dy * (activation_grad(z, act) if act != "none" else 1.0)
    off = 0.0 if act == "none" else 16 * U32 * np.abs(dy) * (1 + (np.abs(z) if act == "silu" else 0.0))
    rounded = off if act == "none" else off + BF16_HALF_STEP * np.abs(u)
    M, N = dy.shape

    def product(a, da, b, K):
        size = np.abs(a) @ np.abs(b)
        extra = 0.0 if act == "none" else da @ np.abs(b)
        return a @ b, (np.ceil(K / 16) + 8) * 2.0 ** -23 * size + 1.01 * extra + TINY

    return (product(u, rounded, w, N), product(u.T, rounded.T if act != "none" else 0.0, x, M),
            (u.sum(0), F32_TOL * np.abs(u).sum(0) + (np.sum(off, 0) if act != "none" else 0.0) + TINY))


def philox(counter, key):
    """Philox 4x32 of ten rounds (Salmon, Moraes, Dror and Shaw, 2011) on arrays of 32-bit words."""
    c, k = [np.asarray(v, dtype=np.uint64) for v in counter], [int(v) for v in key]
    w32, mask = np.uint64(32), np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> w32) ^ c[1] ^ np.uint64(k[0]), b & mask, (a >> w32) ^ c[3] ^ np.uint64(k[1]), a & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_keep(seed, offset, p, first, n):
    """Which of elements first .. first + n - 1 are kept."""
    i = np.arange(first, first + n, dtype=np.uint64)
    block, mask = i >> np.uint64(2), np.uint64(0xFFFFFFFF)
    words = philox((block & mask, block >> np.uint64(32), np.full_like(block, offset & 0xFFFFFFFF),
                    np.full_like(block, offset >> 32)), (seed & 0xFFFFFFFF, seed >> 32))
    word = np.choose((i & np.uint64(3)).astype(np.int64), words)
    return word >= np.uint64(int(np.rint(p * 2.0 ** 32)))


def dropout(x, r, keep, p):
    y = np.where(keep, x / (1.0 - p) if p < 1 else 0.0, 0.0)
    tol = 4 * U32 * (np.abs(y) + (np.abs(r) if r is not None else 0.0)) + TINY
    return (y + r if r is not None else y), tol
