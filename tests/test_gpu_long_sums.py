"""Gradients of what is broadcast over the rows (gamma, bias), added up over very many rows of terms of one sign, whose
rounding must not pile up.

Tolerance: a chain of n equal terms in FP32 is off by at most n / 2 half steps, n / 2 * 2^-24 of the sum.  The sums go in
chains of up to 512 rows, of up to 32 rows' threads and of up to 256 parts with the total carried, and a tree of 5:
(512 + 32 + 256 + 10) / 2 * 2^-24 = 2.4e-5, and 2^-23 for the term itself.  (One chain of 10^4 such terms is off by up to 1.5e-4.)
SiLU's derivative is off by 16 (1 + |z|) * 2^-24 of dy, 1.9e-6 here."""
import numpy as np
import pytest
import torch

import operator_refs as oref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
TOL = 2.5e-5


@pytest.mark.parametrize("M,C", [(1 << 27, 8), (1 << 25, 7), (1 << 22, 1032), (1 << 22, 1031), (1 << 18, 8200), (1 << 17, 16391)])
def test_gamma_gradient_over_very_many_rows(M, C):
    """Rows of 8 lanes, of one warp, of all warps in both kernels that stream rows; longer ones by column."""
    import cnn_convolution_implicit_gb300 as cg
    h = torch.ones(M, C, device="cuda", dtype=BF16)
    rstd = torch.full((M,), 0.1, device="cuda")
    _, dgamma = cg.rms_norm_backward(h, h, rstd)
    want = M * float(np.float32(0.1))
    assert float((dgamma.double() - want).abs().max()) <= TOL * want


@pytest.mark.parametrize("M,N", [(1 << 27, 17), (1 << 16, 40001), (1 << 18, 32768)])
def test_bias_gradient_over_very_many_rows(M, N):
    import cnn_convolution_implicit_gb300 as cg
    z = torch.full((M, N), 0.75, device="cuda", dtype=BF16)
    dy = torch.full((M, N), 0.3, device="cuda", dtype=BF16)
    _, _, dbias = cg.LinearPlan(M, N, 8, "silu").backward(dy, z=z, need=(False, False, True))
    want = M * float(dy[0, 0]) * float(oref.activation_grad(np.array(0.75), "silu"))
    assert float((dbias.double() - want).abs().max()) <= (TOL + 1.9e-6) * want
    if N == 17:  # the products' launch joins the parts instead
        x = torch.zeros(M, 8, device="cuda", dtype=BF16)
        _, _, again = cg.linear_backward(dy, x, torch.zeros(N, 8, device="cuda", dtype=BF16), z, "silu")
        assert torch.equal(again, dbias)


@pytest.mark.parametrize("M,C", [(304 * 8 * 512 + 1, 7), (304 * 32 * 512 + 1, 8), (304 * 512 + 1, 1031), (304 * 512 + 1, 1032), (3 * 304 * 512 - 7, 1025)])
def test_every_row_in_several_rounds(M, C):
    """Just past one round of CTAs, and in three: dx as for the rows by themselves, in its own buffer and over dy, dgamma as in 64
    bits (of rows that a CTA of 152 SMs' rounds takes)."""
    import cnn_convolution_implicit_gb300 as cg
    g = torch.Generator(device="cuda").manual_seed(M)
    dy, h = (torch.randn(M, C, device="cuda", generator=g).to(BF16) for _ in range(2))
    rstd, gamma = torch.rand(M, device="cuda", generator=g) + 0.5, torch.rand(C, device="cuda", generator=g)
    dx, dgamma = cg.rms_norm_backward(dy, h, rstd, gamma, h)
    want, size, step = torch.zeros(C, device="cuda", dtype=torch.float64), torch.zeros(C, device="cuda", dtype=torch.float64), 50001
    for m in range(0, M, step):
        part = slice(m, min(m + step, M))
        alone, _ = cg.rms_norm_backward(dy[part].clone(), h[part].clone(), rstd[part].clone(), gamma, h[part].clone())
        assert torch.equal(alone, dx[part])
        terms = dy[part].double() * h[part].double() * rstd[part].double()[:, None]
        want += terms.sum(0)
        size += terms.abs().sum(0)
    assert torch.all((dgamma.double() - want).abs() <= TOL * size)
    again, dgamma2 = cg.RmsNormPlan(M, C).backward(dy, h, rstd, gamma, h, dx=dy)
    assert torch.equal(again, dx) and torch.equal(dgamma2, dgamma)
    assert cg.device_status() == 0
