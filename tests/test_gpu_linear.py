"""Linear layer on the GPU against 64-bit restatements: one row to many, odd sizes, rows off 16 bytes,
every epilogue, gradients against the formula and against differences, bad values, streams, graphs,
autograd, and the residual branch as a whole."""
import numpy as np
import pytest
import torch

import operator_refs as oref
import row_refs as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    x, r, dy = (torch.randn(M, n, generator=g).to(BF16) for n in (K, N, N))
    w = (torch.randn(N, K, generator=g) / K ** 0.5).to(BF16)
    return x, w, torch.randn(N, generator=g), r, dy


SIZES = [
    # M, N, K
    (1, 1, 1), (1, 17, 5), (1, 4096, 1024), (2, 300, 4096), (3, 1, 64), (4, 1000, 2052), (5, 64, 48), (8, 128, 1000), (9, 40, 16),
    (16, 512, 512), (17, 200, 4104), (31, 77, 333), (32, 256, 2048), (33, 130, 264), (48, 96, 640), (64, 256, 96), (65, 4096, 512),
    (127, 128, 64), (128, 128, 128), (129, 257, 127), (200, 320, 320), (256, 2048, 1024), (301, 777, 1000), (513, 512, 256),
    (1000, 96, 2048), (1000, 1003, 72), (2000, 2050, 520), (3136, 512, 256), (5000, 1000, 200), (40000, 64, 72), (7, 20000, 128),
    # each tile, whole and with its K shared, rows of y on and off 16 bytes
    (443, 2728, 36), (4603, 271, 32), (42, 432, 10952), (37, 3206, 1835), (4785, 1624, 40), (4639, 1956, 32), (130, 3504, 7040),
    (3652, 129, 5960), (34, 34, 1089), (62, 32, 1072), (35, 1455, 4623), (37, 37, 1658), (39, 32, 2599), (1300, 325, 105),
    # the K of a tile shared by two, four, eight CTAs that join it, by three that leave parts; few rows with a long odd K
    (4714, 50, 1664), (4683, 48, 2688), (2127, 36, 921), (42, 1664, 848), (147, 1380, 1344), (34, 2376, 2096), (267, 3492, 7581),
    (4662, 32, 7376), (148, 3232, 2840), (3362, 135, 3305), (41, 32, 6584),
    (931, 1280, 336), (132, 3400, 5392), (38, 2912, 2587), (39, 1392, 3928), (40, 2476, 2166), (276, 3490, 209), (2732, 372, 2488), (264, 2480, 3152),
    (3664, 68, 1352), (1646, 75, 2488), (4638, 50, 7803), (2, 100, 3005),
]

GRAD_SIZES = [(1, 1, 1), (1, 520, 264), (3, 33, 70), (20, 96, 160), (64, 1000, 520), (77, 264, 520), (301, 777, 1000),
              (1000, 96, 48), (129, 257, 127), (2000, 512, 256), (5000, 64, 40), (300, 1024, 2048), (20000, 130, 72),
              # each tile, whole, with the K of dx, of dw or of both shared
              (49, 48, 5304), (39, 32, 6635), (4210, 32, 226), (34, 1984, 518), (705, 33, 8624), (758, 33, 8748),
              (2246, 57, 2792), (58, 3120, 1922), (1198, 36, 32), (34, 1216, 36), (2549, 3552, 39), (1397, 52, 42),
              (37, 2068, 440), (4648, 32, 3238), (3740, 32, 3824), (1925, 40, 43), (41, 2244, 36), (35, 1704, 48), (2256, 34, 32), (5647, 9421, 8),
              (90, 2040, 16), (35, 399, 2765), (1943, 47, 970), (2887, 36, 1088), (33, 2132, 856), (885, 3524, 466), (988, 3024, 664)]


@pytest.mark.parametrize("size", SIZES)
def test_forward(size):
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    x, w, b, r, _ = _inputs(M, N, K, M + 3 * N + K)
    canvas = torch.full((2, M * N + 64), 7.0, device="cuda", dtype=BF16)
    y, z = (c[:M * N].view(M, N) for c in (canvas[0], canvas[1]))
    if canvas[1].data_ptr() % 16:
        z = torch.empty(M, N, device="cuda", dtype=BF16)
    plan = cg.LinearPlan(M, N, K, "silu")
    plan.forward(x.cuda(), w.cuda(), b.cuda(), r.cuda(), y=y, z=z)
    (want, tol), (want_z, tol_z) = ref.linear(_np(x), _np(w), _np(b), _np(r), "silu")
    oref.check(_np(y), want, tol, True, "y")
    oref.check(_np(z), want_z, tol_z, True, "z")
    assert torch.all(canvas[:, M * N:] == 7.0)
    y = cg.linear(x.cuda(), w.cuda())
    (want, tol), _ = ref.linear(_np(x), _np(w), None, None, "none")
    oref.check(_np(y), want, tol, True, "plain y")
    assert plan.device_status() == 0 and cg.device_status() == 0


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("size", [(1, 96, 160), (3, 97, 100), (20, 96, 160), (20, 95, 101), (140, 200, 136), (140, 203, 130), (600, 512, 520),
                                  (140, 200, 2100), (140, 203, 2100)])
def test_every_epilogue(size, act):
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    x, w, b, r, _ = _inputs(M, N, K, 5)
    for bias in (None, b):
        for res in (None, r):
            for with_z in (False, True):
                z = torch.empty(M, N, device="cuda", dtype=BF16) if with_z else None
                y = cg.linear(x.cuda(), w.cuda(), None if bias is None else bias.cuda(), act,
                              None if res is None else res.cuda(), z=z)
                (want, tol), (want_z, tol_z) = ref.linear(_np(x), _np(w), None if bias is None else _np(bias),
                                                          None if res is None else _np(res), act)
                oref.check(_np(y), want, tol, True, "y")
                if with_z:
                    oref.check(_np(z), want_z, tol_z, True, "z")


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("size", GRAD_SIZES)
def test_backward(size, act):
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    x, w, b, _, dy = _inputs(M, N, K, 7 * M + N + K)
    z = None if act == "none" else torch.from_numpy(ref.linear(_np(x), _np(w), _np(b), None, act)[1][0]).to(BF16)
    zc = None if z is None else z.cuda()
    canvas = torch.full((M * K + 64,), 7.0, device="cuda", dtype=BF16)
    plan = cg.LinearPlan(M, N, K, act)
    dx, dw, db = plan.backward(dy.cuda(), x.cuda(), w.cuda(), zc, dx=canvas[:M * K].view(M, K))
    want = ref.linear_backward(_np(dy), _np(x), _np(w), None if z is None else _np(z), act)
    for got, (value, tol), bf16, what in zip((dx, dw, db), want, (True, True, False), ("dx", "dw", "dbias")):
        oref.check(_np(got), value, tol, bf16, what)
    assert torch.all(canvas[M * K:] == 7.0)
    # each by itself, and the functional form, give the same bits
    one = cg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), zc, act)
    for i, (got, name) in enumerate(zip((dx, dw, db), ("dx", "dw", "dbias"))):
        assert torch.equal(one[i], got), name
        need = tuple(j == i for j in range(3))
        alone = plan.backward(dy.cuda(), x.cuda() if i == 1 else None, w.cuda() if i == 0 else None, zc, need=need)
        assert torch.equal(alone[i], got) and all(alone[j] is None for j in range(3) if j != i)
    assert plan.device_status() == 0 and cg.device_status() == 0


@pytest.mark.parametrize("M", [1, 20, 300])
def test_against_differences(M):
    """The product is linear in each operand: (f(x + d) - f(x)) . dy is dx . d up to the roundings of the
    two results to BF16 (2^-8 of them each) and of dx."""
    import cnn_convolution_implicit_gb300 as cg
    N, K = 200, 120
    x, w, b, _, dy = _inputs(M, N, K, 17)
    d = torch.randn(M, K, generator=torch.Generator().manual_seed(4)).to(BF16)
    moved = (x.float() + d.float()).to(BF16)
    step = moved.double() - x.double()
    y0, y1 = _np(cg.linear(x.cuda(), w.cuda(), b.cuda())), _np(cg.linear(moved.cuda(), w.cuda(), b.cuda()))
    dx, dw, _ = cg.linear_backward(dy.cuda(), x.cuda(), w.cuda())
    g = _np(dy)
    tol = 1.1 * 2.0 ** -8 * ((np.abs(y0) + np.abs(y1)) * np.abs(g)).sum() + 2.0 ** -8 * np.abs(_np(dx) * step.numpy()).sum()
    assert abs(((y1 - y0) * g).sum() - (_np(dx) * step.numpy()).sum()) <= tol
    dwt = torch.randn(N, K, generator=torch.Generator().manual_seed(5)).mul(0.1).to(BF16)
    moved = (w.float() + dwt.float()).to(BF16)
    step = (moved.double() - w.double()).numpy()
    y1 = _np(cg.linear(x.cuda(), moved.cuda(), b.cuda()))
    tol = 1.1 * 2.0 ** -8 * ((np.abs(y0) + np.abs(y1)) * np.abs(g)).sum() + 2.0 ** -8 * np.abs(_np(dw) * step).sum()
    assert abs(((y1 - y0) * g).sum() - (_np(dw) * step).sum()) <= tol


@pytest.mark.parametrize("M", [1, 4, 20, 60, 200])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_row_and_column(value, M):
    import cnn_convolution_implicit_gb300 as cg
    N, K = 200, 328
    x, w, b, r, dy = _inputs(M, N, K, 3)
    clean = cg.linear(x.cuda(), w.cuda(), b.cuda(), "silu", r.cuda())
    bad = w.clone()
    bad[77, 5] = value
    y = cg.linear(x.cuda(), bad.cuda(), b.cuda(), "silu", r.cuda())
    cols = [n for n in range(N) if n != 77]
    assert torch.equal(y[:, cols], clean[:, cols])
    assert not torch.any(torch.isfinite(y[:, 77]) & (x[:, 5].cuda() > 0))
    if M > 1:
        bad = x.clone()
        bad[M // 2, 300] = value
        y = cg.linear(bad.cuda(), w.cuda(), b.cuda(), "silu", r.cuda())
        rows = [m for m in range(M) if m != M // 2]
        assert torch.equal(y[rows], clean[rows])
    dx, dw, db = cg.linear_backward(dy.cuda(), x.cuda(), w.cuda())
    dy[M // 2, 9] = value
    dx2, dw2, db2 = cg.linear_backward(dy.cuda(), x.cuda(), w.cuda())
    rows, cols = [m for m in range(M) if m != M // 2], [n for n in range(N) if n != 9]
    assert torch.equal(dx2[rows], dx[rows]) and torch.equal(dw2[cols], dw[cols]) and torch.equal(db2[cols], db[cols])
    assert not torch.isfinite(db2[9])


@pytest.mark.parametrize("size", [(1, 256, 512), (20, 256, 512), (70, 101, 203), (300, 777, 512), (2000, 512, 256),
                                  (1000, 96, 2048), (2127, 36, 921), (35, 1455, 4623)])
def test_residual_in_place(size):
    import cnn_convolution_implicit_gb300 as cg
    x, w, b, r, _ = (t.cuda() for t in _inputs(*size, 31))
    y = cg.linear(x, w, b, "relu", r)
    over = r.clone()
    assert cg.linear(x, w, b, "relu", over, y=over) is over and torch.equal(over, y)


@pytest.mark.parametrize("size", [(1, 256, 512), (20, 256, 512), (70, 101, 203), (300, 777, 512), (2000, 512, 256), (513, 2048, 1024)])
def test_side_stream_graph_and_repeat(size):
    import cnn_convolution_implicit_gb300 as cg
    M, N, K = size
    x, w, b, r, dy = (t.cuda() for t in _inputs(M, N, K, 41))
    z = torch.empty(M, N, device="cuda", dtype=BF16)
    y = cg.linear(x, w, b, "silu", r, z=z)
    grads = cg.linear_backward(dy, x, w, z, "silu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = cg.linear(x, w, b, "silu", r, stream=side)
    grads2 = cg.linear_backward(dy, x, w, z, "silu", stream=side)
    y3 = cg.linear(x, w, b, "silu", r)      # at the same time
    grads3 = cg.linear_backward(dy, x, w, z, "silu")
    torch.cuda.synchronize()
    for got in ([y2, *grads2], [y3, *grads3]):
        assert all(torch.equal(p, q) for p, q in zip([y, *grads], got))
    graph, x4 = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        y4 = cg.linear(x4, w, b, "silu", r)
        grads4 = cg.linear_backward(dy, x4, w, z, "silu")
    x4.copy_(x)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip([y, *grads], [y4, *grads4]))
    assert cg.device_status() == 0


@pytest.mark.parametrize("act,shape", [("none", (2, 5, 24)), ("relu", (3, 40)), ("silu", (2, 3, 7, 33))])
def test_gradients_are_recorded(act, shape):
    import cnn_convolution_implicit_gb300 as cg
    K, N = shape[-1], 50
    M = int(np.prod(shape[:-1]))
    x, w, b, r, dy = _inputs(M, N, K, 51)
    leaves = [t.cuda().requires_grad_(True) for t in (x.view(shape), w, b, r.view(shape[:-1] + (N,)))]
    y = cg.linear(leaves[0], leaves[1], leaves[2], act, leaves[3])
    assert y.shape == shape[:-1] + (N,)
    y.backward(dy.cuda().view(y.shape))
    z = torch.empty(M, N, device="cuda", dtype=BF16)
    cg.linear(x.cuda(), w.cuda(), b.cuda(), act, z=z)
    want = cg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z, act)
    for leaf, value in zip(leaves, [*want, dy.cuda()]):
        assert torch.equal(leaf.grad, value.view(leaf.shape))
    # a gradient for some of them alone, from a gradient that is not contiguous, on another stream
    w2 = w.cuda().requires_grad_(True)
    y = cg.linear(x.cuda().view(shape), w2, b.cuda(), act)
    wide = torch.zeros(*y.shape[:-1], 2 * N, device="cuda", dtype=BF16)
    wide[..., ::2] = dy.cuda().view(y.shape)
    y.backward(wide[..., ::2])
    assert torch.equal(w2.grad, want[1])
    with pytest.raises(ValueError):
        cg.linear(leaves[0], leaves[1], y=torch.empty_like(y))
    with torch.no_grad():
        assert not cg.linear(leaves[0], leaves[1]).requires_grad


def test_refusals():
    import cnn_convolution_implicit_gb300 as cg
    x, w, b, r, dy = (t.cuda() for t in _inputs(6, 8, 16, 61))
    plan = cg.LinearPlan(6, 8, 16, "relu")
    for bad in (dict(x=x.float()), dict(x=x[:5]), dict(w=w.t()), dict(w=w.float()), dict(bias=b[:7]), dict(bias=b.to(BF16)),
                dict(residual=r[:5]), dict(residual=r.float()), dict(y=r.float()), dict(z=r.float()), dict(x=x.cpu()), dict(w=w.cpu())):
        with pytest.raises(ValueError):
            plan.forward(**dict(dict(x=x, w=w), **bad))
    for bad in (dict(dy=dy.float()), dict(x=None), dict(w=None), dict(z=None), dict(dx=x.float()), dict(dw=w.t()), dict(dbias=b[:3]),
                dict(dx=x, need=(False, True, True))):
        with pytest.raises(ValueError):
            plan.backward(**dict(dict(dy=dy, x=x, w=w, z=r), **bad))
    with pytest.raises(cg.ConvError):
        plan.backward(dy, z=r, need=(False, False, False))
    with pytest.raises(ValueError):
        cg.linear(x, w[:, :8])
    with pytest.raises(cg.ConvError):
        cg.linear(x[:0], w)
    with pytest.raises(cg.ConvError):  # a base off 16 bytes
        cg.linear(torch.ones(17, device="cuda", dtype=BF16)[1:].view(1, 16), w)


def test_residual_branch():
    """Product, dropout with the residual, norm: a branch in training, its gradients through autograd
    against the same operators called one by one; and in serving, norm to 8 bits and 8-bit product."""
    import cnn_convolution_implicit_gb300 as cg
    M, C, F = 300, 264, 520
    x, w1, b1, _, _ = _inputs(M, F, C, 71)
    _, w2, b2, r, dy = _inputs(M, C, F, 72)
    gamma = torch.randn(C, generator=torch.Generator().manual_seed(73)) * 0.1 + 1
    state = torch.tensor([5, 6], device="cuda")
    leaves = [t.cuda().requires_grad_(True) for t in (x, w1, b1, w2, b2, gamma)]

    def branch(x, w1, b1, w2, b2, gamma):
        n = cg.rms_norm(x, gamma)
        f = cg.linear(n, w1, b1, "silu")
        return cg.dropout(cg.linear(f, w2, b2), 0.2, state, residual=x)

    y = branch(*leaves)
    y.backward(dy.cuda())
    X, W1, B1, W2, B2, G = (t.detach() for t in leaves)
    rstd, z = torch.empty(M, device="cuda"), torch.empty(M, F, device="cuda", dtype=BF16)
    n = cg.rms_norm(X, G, rstd=rstd)
    f = cg.linear(n, W1, B1, "silu", z=z)
    assert torch.equal(cg.dropout(cg.linear(f, W2, B2), 0.2, state, residual=X), y)
    d = cg.dropout_backward(dy.cuda(), 0.2, state)
    df, dw2, db2 = cg.linear_backward(d, f, W2)
    dn, dw1, db1 = cg.linear_backward(df, n, W1, z, "silu")
    dx, dg = cg.rms_norm_backward(dn, X, rstd, G, dh=dy.cuda())
    for leaf, value in zip(leaves[1:], (dw1, db1, dw2, db2, dg)):
        assert torch.equal(leaf.grad, value)
    # autograd adds the two gradients of x after rounding each to BF16; the call with dh rounds once
    assert torch.all((leaves[0].grad.float() - dx.float()).abs() <= 2.0 ** -7 * (dx.float().abs() + dy.cuda().float().abs()) + 1e-30)
    # against the definitions in 64 bits: five roundings to BF16 on the way, each 2^-8 at most
    xd = _np(x)
    nd = xd / np.sqrt((xd ** 2).mean(1, keepdims=True) + 1e-6) * _np(gamma)
    zd = nd @ _np(w1).T + _np(b1)
    od = (zd / (1 + np.exp(-zd))) @ _np(w2).T + _np(b2)
    keep = ref.dropout_keep(5, 6, 0.2, 0, M * C).reshape(M, C)
    want = xd + np.where(keep, od / 0.8, 0.0)
    assert np.linalg.norm(_np(y) - want) <= 5 * 2.0 ** -8 * np.linalg.norm(want)
    # serving
    wq, ws = cg.quantize_rows(w1.cuda())
    q, scale, h = cg.rms_norm_int8(X, G, residual=r.cuda())
    y8 = cg.int8_matmul(q, scale, wq, ws, b1.cuda())
    want, tol = oref.int8_product(q.cpu().numpy(), scale.cpu().numpy(), wq.cpu().numpy(), ws.cpu().numpy(), b1.numpy(), "none")
    oref.check(_np(y8), want, tol, True, "8-bit product")
    one = cg.linear(h[:1], W1, B1, "silu")
    (want, tol), _ = ref.linear(_np(h[:1]), _np(w1), _np(b1), None, "silu")
    oref.check(_np(one), want, tol, True, "one token")


def test_arguments_that_nobody_else_holds():
    """A caller's temporaries live until the launch: their memory is not given to the call's own buffers (rows to
    lay out, parts of K, results)."""
    import cnn_convolution_implicit_gb300 as cg
    for M, N, K in ((129, 257, 127), (70, 512, 4096), (5, 100, 60)):
        x, w, b, r, dy = _inputs(M, N, K, 91)
        want = cg.linear(x.cuda(), w.cuda(), b.cuda(), "silu", r.cuda())
        keep = [t.cuda() for t in (x, w, b, r, dy)]
        assert torch.equal(cg.linear(*keep[:3], "silu", keep[3]), want)
        for _ in range(3):
            assert torch.equal(cg.linear(*(t.clone() for t in keep[:3]), "silu", keep[3].clone()), want)
            torch.cuda.empty_cache()
        grads = cg.linear_backward(keep[4], keep[0], keep[1], want, "silu")
        again = cg.linear_backward(keep[4].clone(), keep[0].clone(), keep[1].clone(), want.clone(), "silu")
        assert all(torch.equal(p, q) for p, q in zip(grads, again))


def test_output_past_2_31_elements():
    import cnn_convolution_implicit_gb300 as cg
    for N in (8192, 8191):          # by bulk stores and by elements
        M = (1 << 31) // N + 300
        x, w, b, _, _ = _inputs(300, N, 64, 101)
        xs = torch.zeros(M, 64, device="cuda", dtype=BF16)
        xs[-300:] = x.cuda()
        y = cg.linear(xs, w.cuda(), b.cuda(), "relu")
        (want, tol), _ = ref.linear(_np(x), _np(w), _np(b), None, "relu")
        oref.check(_np(y[-300:]), want, tol, True, "y")
        assert torch.equal(y[0], torch.relu(b.cuda()).to(BF16)) and torch.equal(y[M // 2], y[0])
        # gradients of as many values: rows of zeros but for the last 300
        y.zero_()
        y[-300:] = torch.randn(300, N, generator=torch.Generator().manual_seed(7)).to(BF16).cuda()
        dy = y[-300:].cpu()
        dx, dw, db = cg.linear_backward(y, xs, w.cuda())
        (wx, tx), (ww, tw), (wb, tb) = ref.linear_backward(_np(dy), _np(x), _np(w), None, "none")
        oref.check(_np(dx[-300:]), wx, tx, True, "dx")
        oref.check(_np(dw), ww, tw, True, "dw")
        oref.check(_np(db), wb, tb, False, "dbias")
        assert not torch.any(dx[:1000])
        del y, dx


def test_a_captured_training_step():
    """Forward and backward of a whole branch in one graph, its plans made inside the capture, replayed on new inputs:
    the same as eager steps."""
    import cnn_convolution_implicit_gb300 as cg
    M, C, F = 150, 136, 264
    x0, w1, b1, _, _ = _inputs(M, F, C, 111)
    _, w2, b2, _, dy0 = _inputs(M, C, F, 112)
    params = [t.cuda().requires_grad_(True) for t in (w1, b1, w2, b2, torch.ones(C))]
    x, dy = x0.cuda().requires_grad_(True), dy0.cuda()
    state = torch.tensor([1, 0], device="cuda")

    def step(x, dy):
        n = cg.rms_norm(x, params[4])
        y = cg.dropout(cg.linear(cg.linear(n, params[0], params[1], "silu"), params[2], params[3]), 0.1, state, residual=x)
        return torch.autograd.grad(y, [x, *params], dy)

    side = torch.cuda.Stream()          # torch's warm-up; other shapes, so that the capture makes its own plans
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x[:40].detach().requires_grad_(True), dy[:40])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step(x, dy)
        state[1] += 1
    for offset in range(2):
        fresh = torch.randn(M, C, generator=torch.Generator().manual_seed(offset)).to(BF16).cuda()
        with torch.no_grad():
            x.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        got = [g.clone() for g in grads]
        state.copy_(torch.tensor([1, offset]))
        want = step(fresh.requires_grad_(True), dy)
        state[1] += 1
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert cg.device_status() == 0


def test_threads():
    """One cached plan, called from several threads with their own streams: each gets the bits of a call by itself."""
    import threading
    import cnn_convolution_implicit_gb300 as cg
    x, w, b, r, dy = (t.cuda() for t in _inputs(140, 200, 2100, 131))
    want = (cg.linear(x, w, b, "none", r), *cg.linear_backward(dy, x, w), cg.rms_norm(x), *cg.rms_norm_int8(x))
    torch.cuda.synchronize()
    wrong = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = (cg.linear(x, w, b, "none", r), *cg.linear_backward(dy, x, w), cg.rms_norm(x), *cg.rms_norm_int8(x))
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(p, q) for p, q in zip(want, got)):
                    wrong.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and cg.device_status() == 0


def test_two_streams_at_once():
    """Products that share a K and norms that join parts, on two streams at the same time, many times over."""
    import cnn_convolution_implicit_gb300 as cg
    x, w, b, r, dy = (t.cuda() for t in _inputs(130, 250, 5000, 121))
    h, gamma = torch.randn(3000, 1003, device="cuda").to(BF16), torch.ones(1003, device="cuda")
    rstd = torch.rand(3000, device="cuda") + 0.5

    def work():
        return [cg.linear(x, w, b, "silu", r), *cg.linear_backward(dy, x, w), *cg.rms_norm_backward(h, h, rstd, gamma),
                cg.rms_norm(h, gamma, h)[0]]

    want = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            got.append(work())
    torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(p, q) for p, q in zip(want, one))
