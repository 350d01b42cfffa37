"""The linear layer's gradients against the product of the rounded u: where an activation's u = dy act'(z) is rounded
to BF16 for dx and dw, the reference rounds it too, so that a row, a granule or a value of u in the wrong place stands out.

Tolerance: the kernel's u is off by 16 (1 + |z|) * 2^-24 of |dy| with SiLU (not at all with ReLU, a factor of 0 or 1).  Rounding is
monotone, so its BF16 lies between those of u less and u plus that much: nearly always one value, else the distance of the two is
allowed for that element.  The product's own tolerance is row_refs'."""
import numpy as np
import pytest
import torch

import operator_refs as oref
import row_refs as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
# M, N, K: u laid out in 16-byte vectors (N % 8 = 0), 8, 4 and 2 bytes; one strip of columns and many, more rows than a batch, several
# parts of rows; dx and dw whole and with their K shared
SIZES = [(1, 8, 16), (3, 520, 264), (64, 1000, 520), (301, 777, 1000), (1000, 96, 48), (2000, 512, 256), (5000, 64, 40), (300, 1024, 2048),
         (4099, 2056, 72), (20000, 130, 72), (700, 1028, 320), (129, 257, 127), (35, 4096, 96), (9000, 320, 24)]


def _np(t):
    return t.detach().double().cpu().numpy()


def _bf16(v):
    return torch.from_numpy(np.ascontiguousarray(v)).float().to(BF16).double().numpy()


def _reference(dy, x, w, z, act):
    u = dy * oref.activation_grad(z, act)
    off = 16 * ref.U32 * np.abs(dy) * (1 + np.abs(z)) if act == "silu" else 0.0
    low, high = _bf16(u - off), _bf16(u + off)
    rounded, spread = _bf16(u), high - low
    assert (spread > 0).mean() < 0.02  # the allowance is an exception

    def product(a, da, b, K):
        return a @ b, (np.ceil(K / 16) + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(b)) + 1.01 * (da @ np.abs(b)) + ref.TINY

    return product(rounded, spread, w, dy.shape[1]), product(rounded.T, spread.T, x, dy.shape[0])


@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("size", SIZES)
def test_gradients_of_the_rounded_u(size, act):
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    g = torch.Generator().manual_seed(M + 5 * N + K)
    x, z, dy = (torch.randn(M, n, generator=g).to(BF16) for n in (K, N, N))
    w = (torch.randn(N, K, generator=g) / K ** 0.5).to(BF16)
    dx, dw, _ = cg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z.cuda(), act)
    for got, (want, tol), name in zip((dx, dw), _reference(_np(dy), _np(x), _np(w), _np(z), act), ("dx", "dw")):
        oref.check(_np(got), want, tol, True, name)
    assert cg.device_status() == 0
