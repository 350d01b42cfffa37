"""Host-side: the reference of tests/test_gpu_linear_rounded.py notices a mistake in u, and its allowance is the exception."""
import pytest
import torch

import operator_refs as oref
from test_gpu_linear_rounded import BF16, SIZES, _bf16, _np, _reference


def _inputs(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    x, z, dy = (torch.randn(M, n, generator=g).to(BF16) for n in (K, N, N))
    return _np(x), _np(z), _np(dy), _np((torch.randn(N, K, generator=g) / K ** 0.5).to(BF16))


@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("size", SIZES)
def test_the_reference_holds_for_itself(size, act):
    x, z, dy, w = _inputs(*size, size[0] + 5 * size[1] + size[2])
    u = _bf16(dy * oref.activation_grad(z, act))
    for got, (want, tol) in zip((u @ w, u.T @ x), _reference(dy, x, w, z, act)):
        oref.check(_bf16(got), want, tol, True, "gradient")


def test_a_misplaced_granule_is_seen():
    """Eight values of u exchanged with their neighbours."""
    x, z, dy, w = _inputs(2000, 512, 256, 3)
    u = _bf16(dy * oref.activation_grad(z, "silu"))
    u[700, 64:72], u[700, 72:80] = u[700, 72:80].copy(), u[700, 64:72].copy()
    for got, (want, tol) in zip((u @ w, u.T @ x), _reference(dy, x, w, z, "silu")):
        with pytest.raises(AssertionError, match="above its tolerance"):
            oref.check(_bf16(got), want, tol, True, "gradient")
