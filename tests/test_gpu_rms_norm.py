"""Root-mean-square norm on the GPU against 64-bit restatements: every form (one warp to sixteen a row, rows
longer than they hold), rows on and off 16 bytes, with and without residual, gamma, statistics;
8-bit rows bit for bit; gradients against the formula and against differences; streams, graphs, autograd."""
import numpy as np
import pytest
import torch

import operator_refs as oref
import row_refs as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# M, C: rows in one warp (1, 2, 4 vectors a lane), 4, 8, 16 warps, longer; on and off 16 bytes; one
# element; fewer rows than a CTA takes, more than one round of CTAs
SHAPES = [(1, 1), (3, 2), (5, 8), (2, 7), (9, 256), (4, 255), (33, 500), (7, 512), (5, 1003), (6, 1024), (300, 1000), (3, 1025), (2, 2048),
          (4, 2049), (1, 4096), (9, 4100), (3, 4099), (2, 8192), (3, 8195), (2, 16384), (2, 16383), (2, 16400), (1, 33000), (2, 20001),
          (5000, 40), (4001, 33), (1001, 64), (777, 128), (301, 72), (3, 120)]


def _np(t):
    return t.detach().double().cpu().numpy()


def _rows(M, C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, C, generator=g) * (torch.rand(M, 1, generator=g) * 3 + 0.1)
    return x.to(DTYPES[dtype]), torch.randn(M, C, generator=g).to(DTYPES[dtype]), torch.randn(C, generator=g) * 0.3 + 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype):
    import cnn_convolution_implicit_gb300 as cg
    M, C = shape
    x, r, gamma = _rows(M, C, dtype, M + C)
    canvas = torch.full((M * C + 64,), 7.0, device="cuda", dtype=DTYPES[dtype])
    rstd = torch.empty(M, device="cuda")
    plan = cg.RmsNormPlan(M, C, dtype)
    y, h = plan.forward(x.cuda(), gamma.cuda(), r.cuda(), y=canvas[:M * C].view(M, C), rstd=rstd)
    (want, tol), (want_h, tol_h), want_rstd = ref.rms_forward(_np(x), _np(gamma), _np(r), 1e-6)
    oref.check(_np(y), want, tol, dtype == "bf16", "y")
    oref.check(_np(h), want_h, tol_h, dtype == "bf16", "h")
    oref.check(_np(rstd), want_rstd, ref.F32_TOL * want_rstd, False, "rstd")
    assert torch.all(canvas[M * C:] == 7.0)
    y = cg.rms_norm(x.cuda(), eps=1e-5)
    (want, tol), _, _ = ref.rms_forward(_np(x), 1.0, None, 1e-5)
    oref.check(_np(y), want, tol, dtype == "bf16", "y alone")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype):
    import cnn_convolution_implicit_gb300 as cg
    M, C = shape
    h, dy, gamma = _rows(M, C, dtype, 3 * M + C)
    dh = _rows(M, C, dtype, 5)[1]
    rstd = torch.from_numpy(ref.rms_forward(_np(h), 1.0, None, 1e-6)[2]).float()
    canvas = torch.full((M * C + 64,), 7.0, device="cuda", dtype=DTYPES[dtype])
    plan = cg.RmsNormPlan(M, C, dtype)
    dx, dgamma = plan.backward(dy.cuda(), h.cuda(), rstd.cuda(), gamma.cuda(), dh.cuda(), dx=canvas[:M * C].view(M, C))
    (want, tol), (want_g, tol_g) = ref.rms_backward(_np(dy), _np(h), _np(rstd), _np(gamma), _np(dh))
    oref.check(_np(dx), want, tol, dtype == "bf16", "dx")
    oref.check(_np(dgamma), want_g, tol_g, False, "dgamma")
    assert torch.all(canvas[M * C:] == 7.0)
    alone, none = plan.backward(dy.cuda(), h.cuda(), rstd.cuda(), gamma.cuda(), dh.cuda(), gamma_grad=False)
    assert none is None and torch.equal(alone, dx)
    dx, dgamma = cg.rms_norm_backward(dy.cuda(), h.cuda(), rstd.cuda())
    (want, tol), (want_g, tol_g) = ref.rms_backward(_np(dy), _np(h), _np(rstd), np.ones(C), None)
    oref.check(_np(dx), want, tol, dtype == "bf16", "dx without gamma, dh")
    oref.check(_np(dgamma), want_g, tol_g, False, "dgamma without gamma, dh")


@pytest.mark.parametrize("M", [1, 700, 3001, 70000])
@pytest.mark.parametrize("C", [64, 260, 777])
def test_gamma_gradient_over_many_rows(M, C):
    import cnn_convolution_implicit_gb300 as cg
    h, dy, gamma = _rows(M, C, "bf16", M + C)
    rstd = torch.from_numpy(ref.rms_forward(_np(h), 1.0, None, 1e-6)[2]).float()
    _, dgamma = cg.rms_norm_backward(dy.cuda(), h.cuda(), rstd.cuda(), gamma.cuda())
    _, (want, tol) = ref.rms_backward(_np(dy), _np(h), _np(rstd), _np(gamma), None)
    oref.check(_np(dgamma), want, tol, False, "dgamma")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_int8(shape, dtype):
    """scale within the norm's tolerance, q within one step of the value (half a step, and the norm's
    error of 1e-5 of 127 steps), the row's largest at 127, h as without 8 bits."""
    import cnn_convolution_implicit_gb300 as cg
    M, C = shape
    x, r, gamma = _rows(M, C, dtype, 7 * M + C)
    plan = cg.RmsNormPlan(M, C, dtype)
    canvas = torch.full((M * C + 64,), 99, device="cuda", dtype=torch.int8)
    q, scale, h = plan.forward_int8(x.cuda(), gamma.cuda(), r.cuda(), q=canvas[:M * C].view(M, C))
    (want, tol), _, _ = ref.rms_forward(_np(x), _np(gamma), _np(r), 1e-6)
    top = np.abs(want).max(1)
    oref.check(_np(scale), top / 127, 2e-5 * top / 127 + ref.TINY, False, "scale")
    assert np.all(np.abs(_np(q) - want / (top / 127)[:, None]) <= 0.5 + 127 * 2e-5 * 2)
    assert np.all(np.abs(_np(q)).max(1) == 127) and torch.all(canvas[M * C:] == 99)
    _, h2 = plan.forward(x.cuda(), gamma.cuda(), r.cuda())
    assert torch.equal(h, h2)
    if dtype == "f32":  # the rules of quantize_rows, on the same FP32 values
        y, _ = plan.forward(x.cuda(), gamma.cuda(), r.cuda())
        q2, scale2 = cg.quantize_rows(y)
        assert torch.equal(q, q2) and torch.equal(scale, scale2)
    q3, scale3 = cg.rms_norm_int8(x.cuda(), gamma.cuda())
    (want, _), _, _ = ref.rms_forward(_np(x), _np(gamma), None, 1e-6)
    top = np.abs(want).max(1)
    assert np.all(np.abs(_np(q3) - want / (top / 127)[:, None]) <= 0.5 + 127 * 2e-5 * 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(6, 512), (7, 1003), (3, 5000), (2, 20001)])
def test_buffers_that_are_inputs(shape, dtype):
    """h over the residual; dx over dy or dh."""
    import cnn_convolution_implicit_gb300 as cg
    M, C = shape
    x, r, gamma = (t.cuda() for t in _rows(M, C, dtype, 11))
    plan = cg.RmsNormPlan(M, C, dtype)
    rstd = plan.empty_rstd()
    y, h = plan.forward(x, gamma, r, rstd=rstd)
    over = r.clone()
    y2, h2 = plan.forward(x, gamma, over, h=over)
    assert h2 is over and torch.equal(y, y2) and torch.equal(h, over)
    over = r.clone()
    q, scale, _ = plan.forward_int8(x, gamma, r)
    q2, scale2, _ = plan.forward_int8(x, gamma, over, h=over)
    assert torch.equal(q, q2) and torch.equal(scale, scale2) and torch.equal(h, over)
    dx, dgamma = plan.backward(x, h, rstd, gamma, r)
    for buffer in (0, 1):
        dy, dh = x.clone(), r.clone()
        dx2, dgamma2 = plan.backward(dy, h, rstd, gamma, dh, dx=(dy, dh)[buffer])
        assert torch.equal(dx, dx2) and torch.equal(dgamma, dgamma2)


@pytest.mark.parametrize("C", [64, 1003, 4096, 20001])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_bad_values_stay_in_their_row(value, C):
    import cnn_convolution_implicit_gb300 as cg
    x, r, gamma = _rows(6, C, "bf16", 3)
    clean = cg.rms_norm(x.cuda(), gamma.cuda(), r.cuda())[0]
    x[2, C // 2] = value
    y, h = cg.rms_norm(x.cuda(), gamma.cuda(), r.cuda())
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(y[keep], clean[keep]) and not torch.any(torch.isnan(y[keep]))
    if value != value:
        assert torch.all(torch.isnan(y[2]))
    else:
        assert torch.isnan(y[2, C // 2]) and torch.all(y[2].nan_to_num(0.0) == 0)
    q, scale, _ = cg.rms_norm_int8(x.cuda(), gamma.cuda(), r.cuda())
    assert torch.isnan(scale[2]) and torch.all(q[2] == 0) and not torch.any(torch.isnan(scale[keep]))


def test_rows_of_zeros_and_of_extremes():
    import cnn_convolution_implicit_gb300 as cg
    x = torch.zeros(4, 512, dtype=torch.float32)
    x[1] = 1e-30
    x[2] = 3e38            # its squares pass FP32
    x[3] = torch.finfo(torch.float32).tiny
    y = cg.rms_norm(x.cuda(), eps=1e-6).cpu()
    assert torch.all(y[0] == 0) and torch.all(y[2] == 0)
    assert torch.allclose(y[1], torch.full((512,), 1e-27), rtol=1e-5, atol=0)
    q, scale = cg.rms_norm_int8(x.cuda(), eps=1e-6)
    assert scale[0] == 0 and torch.all(q[0] == 0)
    y = cg.rms_norm(x[:1].cuda(), eps=0.0)   # 0 / 0
    assert torch.all(torch.isnan(y))


def test_the_norm_is_of_the_sum_before_its_rounding():
    import cnn_convolution_implicit_gb300 as cg
    x = torch.full((1, 64), 1.0, dtype=torch.bfloat16)
    r = torch.full((1, 64), 2.0 ** -9, dtype=torch.bfloat16)
    x[0, 0] = 256.0
    y, h = cg.rms_norm(x.cuda(), None, r.cuda())
    (want, tol), _, _ = ref.rms_forward(_np(x), 1.0, _np(r), 1e-6)
    oref.check(_np(y), want, tol, True, "y")
    assert torch.equal(h.cpu(), x)


@pytest.mark.parametrize("dtype,C", [("f32", 96), ("f32", 37), ("bf16", 96)])
def test_gradients_are_recorded(dtype, C):
    """Autograd's gradients are the formula's, with a gradient on either output and on both."""
    import cnn_convolution_implicit_gb300 as cg
    M = 10
    x, r, gamma = _rows(M, C, dtype, 9)
    g = torch.Generator().manual_seed(8)
    dy, dh = (torch.randn(M, C, generator=g).to(DTYPES[dtype]) for _ in range(2))
    for use_y, use_h in ((1, 0), (0, 1), (1, 1)):
        leaves = [t.clone().cuda().requires_grad_(True) for t in (x, r, gamma)]
        y, h = cg.rms_norm(leaves[0], leaves[2], leaves[1])
        loss = (y * dy.cuda()).float().sum() * use_y + (h * dh.cuda()).float().sum() * use_h
        loss.backward()
        want_h = (x.float() + r.float()).to(DTYPES[dtype])
        rstd = ref.rms_forward(_np(x), 1.0, _np(r), 1e-6)[2]
        (want, tol), (want_g, tol_g) = ref.rms_backward(_np(dy) * use_y, _np(want_h), rstd, _np(gamma), _np(dh) * use_h)
        oref.check(_np(leaves[0].grad), want, 2 * tol + 4e-7, dtype == "bf16", "dx")
        assert torch.equal(leaves[0].grad, leaves[1].grad)
        oref.check(_np(leaves[2].grad), want_g, 2 * tol_g + 4e-7, False, "dgamma")
    x1 = x.clone().cuda().requires_grad_(True)
    rstd = torch.empty(M, device="cuda")
    y = cg.rms_norm(x1, rstd=rstd)
    y.backward(dy.cuda())
    (want, tol), _ = ref.rms_backward(_np(dy), _np(x), ref.rms_forward(_np(x), 1.0, None, 1e-6)[2], np.ones(C), None)
    oref.check(_np(x1.grad), want, 2 * tol, dtype == "bf16", "dx alone")
    want = ref.rms_forward(_np(x), 1.0, None, 1e-6)[2]
    oref.check(_np(rstd), want, ref.F32_TOL * want, False, "rstd")
    with pytest.raises(ValueError):
        cg.rms_norm(x1, residual=r.cuda(), h=torch.empty_like(x1))
    with torch.no_grad():
        assert not cg.rms_norm(x1).requires_grad


@pytest.mark.parametrize("shape", [(3, 40), (2, 5003)])
def test_backward_against_differences(shape):
    """f(x + e d) - f(x - e d) over 2 e: e = 1e-3 leaves e^2 of the third derivative, 1e-5 of the
    sum of magnitudes, and the norm's FP32 error over e, 2^-24 / e of them."""
    import cnn_convolution_implicit_gb300 as cg
    M, C = shape
    x, dy, gamma = _rows(M, C, "f32", 21)
    x = x / x.square().mean(1, keepdim=True).sqrt()
    d = torch.randn(M, C, generator=torch.Generator().manual_seed(22))
    rstd = torch.empty(M, device="cuda")
    cg.rms_norm(x.cuda(), gamma.cuda(), rstd=rstd)
    dx, dgamma = cg.rms_norm_backward(dy.cuda(), x.cuda(), rstd, gamma.cuda())
    e = 1e-3

    def f(x, gamma):
        return (_np(cg.rms_norm(x.cuda(), gamma.cuda())) * _np(dy))

    up, down = f(x + e * d, gamma), f(x - e * d, gamma)
    slope, size = (up - down).sum() / (2 * e), np.abs(_np(dx) * _np(d)).sum() + np.abs(up).sum()
    assert abs(slope - (_np(dx) * _np(d)).sum()) <= 2e-4 * size
    dg = torch.randn(C, generator=torch.Generator().manual_seed(23))
    up, down = f(x, gamma + e * dg), f(x, gamma - e * dg)
    slope = (up - down).sum() / (2 * e)
    assert abs(slope - (_np(dgamma) * _np(dg)).sum()) <= 2e-4 * (np.abs(up).sum() + np.abs(_np(dgamma) * _np(dg)).sum())


def test_side_stream_graph_and_repeat():
    import cnn_convolution_implicit_gb300 as cg
    M, C = 37, 1000
    x, r, gamma = (t.cuda() for t in _rows(M, C, "bf16", 30))
    rstd = torch.empty(M, device="cuda")
    y, h = cg.rms_norm(x, gamma, r, rstd=rstd)
    dx, dgamma = cg.rms_norm_backward(x, h, rstd, gamma, r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, h2 = cg.rms_norm(x, gamma, r, stream=side)
    dx2, dgamma2 = cg.rms_norm_backward(x, h, rstd, gamma, r, stream=side)
    q2, s2, _ = cg.rms_norm_int8(x, gamma, r, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(dx, dx2) and torch.equal(dgamma, dgamma2)
    graph, x3 = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        y3, h3 = cg.rms_norm(x3, gamma, r)
        dx3, dgamma3 = cg.rms_norm_backward(x3, h, rstd, gamma, r)
    x3.copy_(x)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y3) and torch.equal(h, h3) and torch.equal(dx, dx3) and torch.equal(dgamma, dgamma3)


def test_shapes_of_any_rank_and_refusals():
    import cnn_convolution_implicit_gb300 as cg
    x = torch.randn(2, 3, 5, 64, device="cuda")
    assert cg.rms_norm(x).shape == x.shape
    q, s = cg.rms_norm_int8(x)
    assert q.shape == x.shape and s.shape == (30,)
    plan = cg.RmsNormPlan(30, 64, "f32", x_shape=x.shape)
    f = torch.ones(64, device="cuda")
    for bad in (dict(x=x.bfloat16()), dict(x=x.transpose(0, 1)), dict(x=x.cpu()), dict(gamma=f[:63]), dict(gamma=f.double()),
                dict(residual=x[:1]), dict(h=torch.empty_like(x)), dict(rstd=f), dict(y=x.bfloat16()),
                dict(residual=x, h=x.bfloat16())):
        with pytest.raises(ValueError):
            plan.forward(**dict(dict(x=x), **bad))
    with pytest.raises(ValueError):
        plan.backward(x, x, f)
    with pytest.raises(ValueError):
        plan.backward(x, x, s, dgamma=f, gamma_grad=False)
    with pytest.raises(ValueError):
        cg.rms_norm(torch.ones(8, device="cuda"))
    with pytest.raises(cg.ConvError):
        cg.rms_norm(torch.ones(0, 8, device="cuda"))
    with pytest.raises(cg.ConvError):  # a base off 16 bytes
        cg.rms_norm(torch.ones(65, device="cuda")[1:].view(1, 64))


def test_rows_past_2_31_elements():
    import cnn_convolution_implicit_gb300 as cg
    M, C = (1 << 31) // 1000 + 5, 1000
    x = torch.zeros(M, C, device="cuda", dtype=torch.bfloat16)
    x[-3:] = torch.randn(3, C, device="cuda").to(torch.bfloat16)
    y = cg.rms_norm(x)
    (want, tol), _, _ = ref.rms_forward(_np(x[-3:]), 1.0, None, 1e-6)
    oref.check(_np(y[-3:]), want, tol, True, "y")
    del y
    rstd = torch.ones(M, device="cuda")
    dx, _ = cg.rms_norm_backward(x, x, rstd)
    (want, tol), _ = ref.rms_backward(_np(x[-3:]), _np(x[-3:]), np.ones(3), np.ones(C), None)
    oref.check(_np(dx[-3:]), want, tol, True, "dx")
