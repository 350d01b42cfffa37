"""The root-mean-square norm's rings in shared memory, used many times over: more groups of rows to a CTA than the ring has
stages, more rows to a stage than the warps take in one turn.  Every value of every output, with and without
residual or dh, each output in a buffer of its own and over its input.  tests/test_rms_ring.py checks on the host that these sizes
do what they are here for."""
import numpy as np
import pytest
import torch

import operator_refs as oref
import row_refs as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# M, C: rows off 16 bytes, a warp each and all warps to one; rows on 16 bytes in 8 and 16 lanes, a warp, all warps
SIZES = [(340000, 33), (200000, 77), (24000, 1003), (3000, 4099), (100000, 64), (60000, 120), (200000, 28), (24000, 1000), (6000, 4096)]


def _np(t):
    return t.detach().double().cpu().numpy()


def _rows(M, C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, C, generator=g) * (torch.rand(M, 1, generator=g) * 3 + 0.1)
    return x.to(DTYPES[dtype]), torch.randn(M, C, generator=g).to(DTYPES[dtype]), torch.randn(C, generator=g) * 0.3 + 1


def _clean():
    import cnn_convolution_implicit_gb300 as cg
    assert cg.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_forward(size, dtype):
    import cnn_convolution_implicit_gb300 as cg
    M, C = size
    x, r, gamma = _rows(M, C, dtype, M + C)
    X, R, G = x.cuda(), r.cuda(), gamma.cuda()
    plan = cg.RmsNormPlan(M, C, dtype)
    rstd, over = plan.empty_rstd(), R.clone()
    y, h = plan.forward(X, G, R, rstd=rstd)
    (want, tol), (want_h, tol_h), want_rstd = ref.rms_forward(_np(x), _np(gamma), _np(r), 1e-6)
    oref.check(_np(y), want, tol, dtype == "bf16", "y")
    oref.check(_np(h), want_h, tol_h, dtype == "bf16", "h")
    oref.check(_np(rstd), want_rstd, ref.F32_TOL * want_rstd, False, "rstd")
    again, _ = plan.forward(X, G, over, h=over)
    assert torch.equal(again, y) and torch.equal(over, h)
    (want, tol), _, _ = ref.rms_forward(_np(x), _np(gamma), None, 1e-6)
    oref.check(_np(plan.forward(X, G)), want, tol, dtype == "bf16", "y alone")
    _clean()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_forward_int8(size, dtype):
    """The tolerances of q and its scale: half a step, and the norm's error of 1e-5 of 127 steps twice over."""
    import cnn_convolution_implicit_gb300 as cg
    M, C = size
    x, r, gamma = _rows(M, C, dtype, 7 * M + C)
    X, R, G = x.cuda(), r.cuda(), gamma.cuda()
    plan = cg.RmsNormPlan(M, C, dtype)
    over = R.clone()
    q, scale, h = plan.forward_int8(X, G, R)
    _, h2 = plan.forward(X, G, R)
    assert torch.equal(h, h2)
    q2, scale2, _ = plan.forward_int8(X, G, over, h=over)
    assert torch.equal(q, q2) and torch.equal(scale, scale2) and torch.equal(over, h)
    for got, s, res in ((q, scale, r), (*plan.forward_int8(X, G), None)):
        (want, _), _, _ = ref.rms_forward(_np(x), _np(gamma), None if res is None else _np(res), 1e-6)
        top = np.abs(want).max(1)
        oref.check(_np(s), top / 127, 2e-5 * top / 127 + ref.TINY, False, "scale")
        assert np.all(np.abs(_np(got) - want / (top / 127)[:, None]) <= 0.5 + 127 * 2e-5 * 2)
    _clean()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_backward(size, dtype):
    import cnn_convolution_implicit_gb300 as cg
    M, C = size
    h, dy, gamma = _rows(M, C, dtype, 3 * M + C)
    dh = _rows(M, C, dtype, 5)[1]
    rstd = torch.from_numpy(ref.rms_forward(_np(h), 1.0, None, 1e-6)[2]).float()
    H, DY, DH, G, S = h.cuda(), dy.cuda(), dh.cuda(), gamma.cuda(), rstd.cuda()
    plan = cg.RmsNormPlan(M, C, dtype)
    dx, dgamma = plan.backward(DY, H, S, G, DH)
    (want, tol), (want_g, tol_g) = ref.rms_backward(_np(dy), _np(h), _np(rstd), _np(gamma), _np(dh))
    oref.check(_np(dx), want, tol, dtype == "bf16", "dx")
    oref.check(_np(dgamma), want_g, tol_g, False, "dgamma")
    for which in (0, 1):
        given = [DY.clone(), DH.clone()]
        dx2, dgamma2 = plan.backward(given[0], H, S, G, given[1], dx=given[which])
        assert torch.equal(dx2, dx) and torch.equal(dgamma2, dgamma)
    assert torch.equal(plan.backward(DY, H, S, G, DH, gamma_grad=False)[0], dx)
    dx, dgamma = plan.backward(DY, H, S, G)
    (want, tol), _ = ref.rms_backward(_np(dy), _np(h), _np(rstd), _np(gamma), None)
    oref.check(_np(dx), want, tol, dtype == "bf16", "dx without dh")
    oref.check(_np(dgamma), want_g, tol_g, False, "dgamma without dh")
    assert torch.equal(plan.backward(DY, H, S, G, gamma_grad=False)[0], dx)
    _clean()
