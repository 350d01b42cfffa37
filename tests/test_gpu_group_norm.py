"""Group norm with an activation on the GPU against 64-bit restatements: forward, backward and
8-bit output over ragged maps, odd channel counts, one-value groups, flat and far-off groups,
NaN and Inf, streams, graphs and repeated runs."""
import numpy as np
import pytest
import torch

import operator_refs as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _make(N, H, W, C, dtype, seed, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, H, W, C, generator=g) * (torch.rand(C, generator=g) + 0.5) + torch.randn(C, generator=g) * offset
    gamma = torch.randn(C, generator=g) * 0.3 + 1.0
    beta = torch.randn(C, generator=g) * 0.3
    return x.to(DT[dtype]), gamma, beta


def _np(t):
    return t.detach().double().cpu().numpy()


def _flat(t):
    a = _np(t)
    return a.reshape(a.shape[0], -1, a.shape[-1])


SHAPES = [
    # N, H, W, C, groups
    (1, 1, 1, 8, 1),        # one pixel
    (1, 1, 1, 16, 16),      # groups of one value: variance 0
    (2, 3, 5, 7, 1),        # odd channels: no vector access
    (3, 7, 3, 30, 5),       # 6 channels a group, rows off 16 bytes in BF16
    (2, 9, 11, 24, 24),     # each channel by itself
    (1, 8, 8, 256, 32),
    (2, 13, 17, 120, 8),    # 15 channels a group: groups end inside vectors
    (5, 16, 16, 64, 2),
    (2, 33, 31, 96, 12),
    (1, 5, 3, 2056, 8),     # wider than one block of threads
    (70, 2, 2, 32, 4),      # many small images
    (1, 96, 100, 64, 8),    # a long map
    (2, 64, 64, 320, 32),   # 10 channels a group
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, act, dtype):
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = shape
    x, gamma, beta = _make(N, H, W, C, dtype, 7 * C + H)
    stats = torch.empty(2, N, G, device="cuda")
    y = cg.group_norm(x.cuda(), G, gamma.cuda(), beta.cuda(), eps=1e-5, act=act, stats=stats)
    want, tol = ref.norm_forward(_flat(x), G, _np(gamma), _np(beta), 1e-5, act)
    ref.check(_flat(y), want, tol, dtype == "bf16", "y")
    mean, rstd = ref.norm_stats(_flat(x), G, 1e-5)
    ref.check(_np(stats[0]), mean, 1e-6 * (1.0 + np.abs(mean)), False, "mean")
    ref.check(_np(stats[1]), rstd, 1e-5 * rstd, False, "rstd")


# Maps that no cluster holds: two passes over pixel ranges, joined in the second (twelve images) or
# by a kernel between them (one image, hundreds of ranges); 40 vectors a pixel: 8-bit rows find
# their magnitude through shared memory.
LARGE = [(1, 200, 210, 64, 8), (12, 190, 200, 32, 4), (2, 250, 130, 320, 32)]

# Small maps of which one CTA holds many groups, and clusters of a dozen CTAs; more clusters than
# the device runs at a time.
HELD = [(40, 7, 7, 320, 20), (160, 5, 3, 104, 13), (20, 14, 14, 512, 32), (4, 96, 96, 64, 4), (160, 28, 28, 96, 8),
        (3, 150, 160, 32, 2), (80, 9, 9, 2048, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", LARGE + HELD)
def test_maps_beyond_a_cluster(shape, dtype):
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = shape
    x, gamma, beta = _make(N, H, W, C, dtype, 13, offset=3.0)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).to(DT[dtype])
    xd, gd, bd = x.cuda(), gamma.cuda(), beta.cuda()
    stats = torch.empty(2, N, G, device="cuda")
    y = cg.group_norm(xd, G, gd, bd, act="silu", stats=stats)
    want, tol = ref.norm_forward(_flat(x), G, _np(gamma), _np(beta), 1e-5, "silu")
    ref.check(_flat(y), want, tol, dtype == "bf16", "y")
    mean, rstd = ref.norm_stats(_flat(x), G, 1e-5)
    ref.check(_np(stats[0]), mean, 1e-6 * (1.0 + np.abs(mean)), False, "mean")
    ref.check(_np(stats[1]), rstd, 1e-5 * rstd, False, "rstd")
    q, scale = cg.group_norm_int8(xd, G, gd, bd, act="silu")
    flat, s = want.reshape(-1, C), _np(scale)
    err = np.abs(_np(q).reshape(-1, C) * s[:, None] - flat)
    assert np.all(err <= 0.5 * s[:, None] * (1 + 128 * ref.U32 * 2) + tol.reshape(-1, C))
    got = cg.group_norm_backward(dy.cuda(), xd, stats, G, gd, bd, act="silu")
    want, tol = ref.norm_backward(_flat(dy), _flat(x), stats.cpu().numpy(), G, _np(gamma), _np(beta), "silu")
    ref.check(_flat(got[0]), want[0], tol[0], dtype == "bf16", "dx")
    ref.check(_np(got[1]), want[1], tol[1], False, "dgamma")
    ref.check(_np(got[2]), want[2], tol[2], False, "dbeta")


@pytest.mark.parametrize("gamma_on,beta_on", [(True, False), (False, True), (False, False)])
def test_forward_without_affine(gamma_on, beta_on):
    import cnn_convolution_implicit_gb300 as cg
    x, gamma, beta = _make(2, 6, 7, 48, "f32", 3)
    y = cg.group_norm(x.cuda(), 6, gamma.cuda() if gamma_on else None, beta.cuda() if beta_on else None, act="silu")
    want, tol = ref.norm_forward(_flat(x), 6, _np(gamma) if gamma_on else np.ones(48),
                                 _np(beta) if beta_on else np.zeros(48), 1e-5, "silu")
    ref.check(_flat(y), want, tol, False, "y")


@pytest.mark.parametrize("shape", [(2, 20, 20, 64, 8), (1, 90, 110, 128, 4), (1, 3, 3, 21, 3)])
@pytest.mark.parametrize("first", ["typical", "outlier"])
def test_forward_far_from_zero(shape, first):
    """Groups whose mean is 1,000 times their spread keep their variance, also where the first
    pixels (a border) lie nowhere near the rest."""
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = shape
    x, gamma, beta = _make(N, H, W, C, "f32", 11)
    x = x + 1000.0
    if first == "outlier":
        x[:, 0] = 0.0
    y = cg.group_norm(x.cuda(), G, gamma.cuda(), beta.cuda())
    want, tol = ref.norm_forward(_flat(x), G, _np(gamma), _np(beta), 1e-5, "none")
    ref.check(_flat(y), want, tol, False, "y")


def test_flat_groups_give_beta():
    import cnn_convolution_implicit_gb300 as cg
    x = torch.full((2, 5, 5, 16), 3.0)
    beta = torch.linspace(-1, 1, 16)
    y = cg.group_norm(x.cuda(), 4, None, beta.cuda())
    assert torch.equal(y.cpu(), beta.expand(2, 5, 5, 16))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("shape", [(2, 6, 6, 32, 4), (2, 4, 4, 21, 3), (2, 80, 80, 64, 4)])
def test_bad_values_stay_in_their_group(value, shape):
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = shape
    x, gamma, beta = _make(N, H, W, C, "f32", 5)
    clean = cg.group_norm(x.cuda(), G, gamma.cuda(), beta.cuda(), act="silu").cpu()
    x[1, 2, 3, 0] = value
    y = cg.group_norm(x.cuda(), G, gamma.cuda(), beta.cuda(), act="silu").cpu()
    cpg = C // G
    assert torch.isnan(y[1, :, :, :cpg]).all()
    assert torch.equal(y[0], clean[0]) and torch.equal(y[1, :, :, cpg:], clean[1, :, :, cpg:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, act, dtype):
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = shape
    x, gamma, beta = _make(N, H, W, C, dtype, 3 * C + W)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(C)).to(DT[dtype])
    stats = torch.empty(2, N, G, device="cuda")
    cg.group_norm(x.cuda(), G, gamma.cuda(), beta.cuda(), act=act, stats=stats)
    got = cg.group_norm_backward(dy.cuda(), x.cuda(), stats, G, gamma.cuda(), beta.cuda(), act=act)
    want, tol = ref.norm_backward(_flat(dy), _flat(x), stats.cpu().numpy(), G, _np(gamma), _np(beta), act)
    ref.check(_flat(got[0]), want[0], tol[0], dtype == "bf16", "dx")
    ref.check(_np(got[1]), want[1], tol[1], False, "dgamma")
    ref.check(_np(got[2]), want[2], tol[2], False, "dbeta")


@pytest.mark.parametrize("act", ["none", "silu"])
def test_backward_against_differences(act):
    """dx, dgamma, dbeta against central differences of the 64-bit forward pass: step 1e-4, so
    the differences themselves are good to about 1e-7 of the loss's third derivative."""
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = 2, 3, 4, 12, 3
    x, gamma, beta = _make(N, H, W, C, "f32", 21)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(9))
    stats = torch.empty(2, N, G, device="cuda")
    cg.group_norm(x.cuda(), G, gamma.cuda(), beta.cuda(), act=act, stats=stats)
    dx, dgamma, dbeta = cg.group_norm_backward(dy.cuda(), x.cuda(), stats, G, gamma.cuda(), beta.cuda(), act=act)
    args = [_flat(x), _np(gamma), _np(beta)]

    def loss(xv, gv, bv):
        return float((ref.norm_forward(xv, G, gv, bv, 1e-5, act)[0] * _flat(dy)).sum())

    rng = np.random.default_rng(4)
    for k, got in enumerate((_flat(dx), _np(dgamma), _np(dbeta))):
        for i in rng.choice(got.size, 12, replace=False):
            moved = []
            for sign in (1, -1):
                v = [a.copy() for a in args]
                v[k].reshape(-1)[i] += sign * 1e-4
                moved.append(loss(*v))
            assert abs((moved[0] - moved[1]) / 2e-4 - got.reshape(-1)[i]) <= 2e-5 * (1.0 + abs(got.reshape(-1)[i]))


def test_backward_without_affine_gradients_to_weights():
    """gamma and beta absent: the gradients that they would have are still the sums."""
    import cnn_convolution_implicit_gb300 as cg
    x, _, _ = _make(2, 5, 6, 32, "f32", 2)
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(1))
    stats = torch.empty(2, 2, 4, device="cuda")
    cg.group_norm(x.cuda(), 4, act="silu", stats=stats)
    got = cg.group_norm_backward(dy.cuda(), x.cuda(), stats, 4, act="silu")
    want, tol = ref.norm_backward(_flat(dy), _flat(x), stats.cpu().numpy(), 4, np.ones(32), np.zeros(32), "silu")
    for g, w, t in zip((_flat(got[0]), _np(got[1]), _np(got[2])), want, tol):
        ref.check(g, w, t, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_int8(shape, act, dtype):
    """One step of q is amax / 127; the FP32 value that was rounded lies within half a step."""
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = shape
    x, gamma, beta = _make(N, H, W, C, dtype, 5 * C + H)
    q, scale = cg.group_norm_int8(x.cuda(), G, gamma.cuda(), beta.cuda(), act=act)
    want, tol = ref.norm_forward(_flat(x), G, _np(gamma), _np(beta), 1e-5, act)
    want, tol = want.reshape(-1, C), tol.reshape(-1, C)
    top, s = np.abs(want).max(1), _np(scale)
    assert q.dtype == torch.int8 and tuple(q.shape) == (N, H, W, C) and tuple(scale.shape) == (N * H * W,)
    assert np.all(np.abs(127.0 * s - top) <= tol.max(1) + 4 * ref.U32 * top)
    err = np.abs(_np(q).reshape(-1, C) * s[:, None] - want)
    assert np.all(err <= 0.5 * s[:, None] * (1 + 128 * ref.U32 * 2) + tol)
    assert np.all(np.abs(_np(q).reshape(-1, C)).max(1)[s > 0] == 127)


def test_forward_int8_bad_group_makes_its_pixels_nan():
    """A NaN group leaves no number in any pixel of its image (each has channels of that group),
    and none of the other image's changes."""
    import cnn_convolution_implicit_gb300 as cg
    x, gamma, beta = _make(2, 6, 6, 32, "bf16", 8)
    clean, cs = cg.group_norm_int8(x.cuda(), 4, gamma.cuda(), beta.cuda())
    x[1, 0, 0, 9] = float("nan")
    q, s = cg.group_norm_int8(x.cuda(), 4, gamma.cuda(), beta.cuda())
    assert torch.isnan(s[36:]).all() and (q[1] == 0).all()
    assert torch.equal(q[0], clean[0]) and torch.equal(s[:36], cs[:36])


@pytest.mark.parametrize("shape", [(2, 9, 11, 96, 12), (16, 64, 64, 64, 8), (1, 150, 160, 256, 32), (1, 7, 5, 21, 7)])
def test_same_inputs_same_bits(shape):
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = shape
    x, gamma, beta = (t.cuda() for t in _make(N, H, W, C, "bf16", 1))
    dy = torch.randn(x.shape, device="cuda").to(torch.bfloat16)

    def once():
        stats = torch.empty(2, N, G, device="cuda")
        y = cg.group_norm(x, G, gamma, beta, act="silu", stats=stats)
        return (y, stats) + cg.group_norm_backward(dy, x, stats, G, gamma, beta, act="silu") + \
            cg.group_norm_int8(x, G, gamma, beta, act="silu")

    first = once()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))


def test_side_stream_and_graph():
    """Inputs made on another stream, the call on a given one, and a captured call replayed on
    new values: each gives the eager call's bits."""
    import cnn_convolution_implicit_gb300 as cg
    x, gamma, beta = (t.cuda() for t in _make(4, 24, 20, 64, "bf16", 6))
    plan = cg.GroupNormPlan(4, 64, 24, 20, 8, "bf16", act="silu")
    want = plan.forward(x, gamma, beta)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = plan.forward(x, gamma, beta, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    dy = torch.randn_like(x)
    y, stats = torch.empty_like(x), plan.empty_stats()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.forward(x, gamma, beta, y=y, stats=stats)
        grads = plan.backward(dy, x, stats, gamma, beta)
    x.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    again = plan.empty_stats()
    assert torch.equal(y, plan.forward(x, gamma, beta, stats=again)) and torch.equal(stats, again)
    for a, b in zip(grads, plan.backward(dy, x, again, gamma, beta)):
        assert torch.equal(a, b)


def test_map_past_2_31_elements():
    """Offsets past 31 bits: the last image of a batch of 2^31 + elements equals itself alone."""
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = 9, 512, 512, 1024, 32
    x = torch.zeros(N, H, W, C, dtype=torch.bfloat16, device="cuda")
    x[-1].normal_()
    y = cg.group_norm(x, G, act="relu")
    alone = cg.group_norm(x[-1:].clone(), G, act="relu")
    assert (y[:-1] == 0).all()
    d = (y[-1].float() - alone[0].float()).abs().max()  # other pixel ranges, so the last bit may differ
    assert float(d) <= 2.0 ** -7 * float(alone.float().abs().max())


def test_binding_refusals():
    import cnn_convolution_implicit_gb300 as cg
    x, gamma, beta = (t.cuda() for t in _make(2, 4, 4, 32, "bf16", 1))
    plan = cg.GroupNormPlan(2, 32, 4, 4, 4)
    with pytest.raises(ValueError):
        plan.forward(x.float(), gamma, beta)                       # type
    with pytest.raises(ValueError):
        plan.forward(x.transpose(1, 2), gamma, beta)               # layout
    with pytest.raises(ValueError):
        plan.forward(x, gamma[:16], beta)                          # shape
    with pytest.raises(ValueError):
        plan.forward(x, gamma.cpu(), beta)                         # device
    with pytest.raises(ValueError):
        plan.backward(x, x, None, gamma, beta)                     # no statistics
    with pytest.raises(ValueError):
        cg.group_norm(x[0], 4)                                     # not NHWC
    with pytest.raises(ValueError):
        cg.group_norm(x, 4, act="gelu")
    with pytest.raises(cg.ConvError):
        cg.group_norm(x, 5)                                        # 32 % 5
    flat = torch.zeros(2 * 4 * 4 * 32 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(cg.ConvError) as e:
        plan.forward(flat[1:1025].view(2, 4, 4, 32), gamma, beta)  # 2 bytes off 16
    assert e.value.status == 3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("shift", [10.0, -10.0])
@pytest.mark.parametrize("shape", [(2, 3, 5, 1, 1), (1, 4, 4, 7, 1), (2, 3, 4, 7, 7), (3, 5, 3, 21, 3), (1, 40, 30, 21, 1)])
def test_forward_int8_odd_channels_far_from_zero(shape, shift, act, dtype):
    """Channels in single accesses: a pixel's scale comes from its own values alone, wherever the
    mean lies (ten spreads from 0 here)."""
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = shape
    x, gamma, beta = _make(N, H, W, C, "f32", 9 * C + H, offset=0.0)
    x = (x + shift).to(DT[dtype])
    q, scale = cg.group_norm_int8(x.cuda(), G, gamma.cuda(), beta.cuda(), act=act)
    want, tol = ref.norm_forward(_flat(x), G, _np(gamma), _np(beta), 1e-5, act)
    want, tol = want.reshape(-1, C), tol.reshape(-1, C)
    top, s, qs = np.abs(want).max(1), _np(scale), _np(q).reshape(-1, C)
    assert np.all(np.abs(127.0 * s - top) <= tol.max(1) + 4 * ref.U32 * top)
    assert np.all(np.abs(qs).max(1)[s > 0] == 127)
    assert np.all(np.abs(qs * s[:, None] - want) <= 0.5 * s[:, None] * (1 + 128 * ref.U32 * 2) + tol)


def _leaf(t, on=True):
    return t.detach().clone().requires_grad_(on)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 9, 7, 64, 8), (1, 40, 30, 21, 3), (4, 56, 56, 64, 4), (1, 8, 8, 256, 32)])
def test_gradients_are_recorded(shape, dtype):
    """group_norm in a graph of operations: the gradients that torch hands back are
    group_norm_backward's, the other branch's are added, and what needs none gets none."""
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = shape
    x, gamma, beta = (t.cuda() for t in _make(N, H, W, C, dtype, 31))
    dy = torch.randn(x.shape, generator=torch.Generator().manual_seed(7)).to(DT[dtype]).cuda()
    stats = torch.empty(2, N, G, device="cuda")
    y = cg.group_norm(x, G, gamma, beta, act="silu", stats=stats)
    want = cg.group_norm_backward(dy, x, stats, G, gamma, beta, act="silu")
    for need in ((True, True, True), (True, False, False), (False, True, False), (False, False, True)):
        a, b, c = _leaf(x, need[0]), _leaf(gamma, need[1]), _leaf(beta, need[2])
        given = torch.empty_like(stats)
        out = cg.group_norm(a, G, b, c, act="silu", stats=given)
        assert out.requires_grad and torch.equal(out, y) and torch.equal(given, stats)
        given.fill_(float("nan"))  # the caller's statistics are the caller's
        out.backward(dy)
        for leaf, on, w in zip((a, b, c), need, want):
            assert (leaf.grad is not None) == on and (not on or torch.equal(leaf.grad, w))
    a = _leaf(x)
    (cg.group_norm(a, G, act="relu") + a).sum().backward()  # no affine; an expanded gradient of ones
    s0 = torch.empty_like(stats)
    cg.group_norm(x, G, act="relu", stats=s0)
    dx = cg.group_norm_backward(torch.ones_like(x), x, s0, G, act="relu")[0]
    assert torch.equal(a.grad, dx + torch.ones_like(x))


def test_gradients_of_odd_layouts_and_streams():
    """A gradient that arrives transposed or off 16 bytes, a call on a given stream, and what cannot
    be recorded."""
    import cnn_convolution_implicit_gb300 as cg
    x, gamma, beta = (t.cuda() for t in _make(2, 6, 6, 32, "bf16", 3))
    dy = torch.randn_like(x)
    stats = torch.empty(2, 2, 4, device="cuda")
    y = cg.group_norm(x, 4, gamma, beta, stats=stats)
    want = cg.group_norm_backward(dy, x, stats, 4, gamma, beta)[0]
    a = _leaf(x)
    cg.group_norm(a, 4, gamma, beta).transpose(1, 2).backward(dy.transpose(1, 2).contiguous())
    assert torch.equal(a.grad, want)
    a, flat = _leaf(x), torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
    off = flat[1:].view(x.shape)
    off.copy_(dy)
    cg.group_norm(a, 4, gamma, beta).backward(off)
    assert torch.equal(a.grad, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = _leaf(x)
    out = cg.group_norm(a, 4, gamma, beta, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    out.backward(dy)
    torch.cuda.synchronize()
    assert torch.equal(out, y) and torch.equal(a.grad, want)
    with torch.no_grad():
        assert not cg.group_norm(_leaf(x), 4, gamma, beta, y=torch.empty_like(x)).requires_grad
    with pytest.raises(ValueError):
        cg.group_norm(_leaf(x), 4, gamma, beta, y=torch.empty_like(x))
    a = _leaf(x.float())
    g = torch.autograd.grad(cg.group_norm(a, 4, act="silu").sum(), a, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        g.sum().backward()  # differentiable once


@pytest.mark.parametrize("shape", [(2, 9, 7, 64, 8), (1, 40, 30, 21, 3), (16, 64, 64, 64, 8)])
def test_dx_alone(shape):
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = shape
    x, gamma, beta = (t.cuda() for t in _make(N, H, W, C, "bf16", 17))
    plan = cg.GroupNormPlan(N, C, H, W, G, "bf16", act="silu")
    stats, dy = plan.empty_stats(), torch.randn_like(x)
    plan.forward(x, gamma, beta, stats=stats)
    dx, dgamma, dbeta = plan.backward(dy, x, stats, gamma, beta, affine_grads=False)
    assert dgamma is None and dbeta is None
    assert torch.equal(dx, plan.backward(dy, x, stats, gamma, beta)[0])
    with pytest.raises(ValueError):
        plan.backward(dy, x, stats, gamma, beta, dgamma=torch.empty_like(gamma), affine_grads=False)


def test_channels_past_65535_blocks():
    """An odd number of channels, 65,536 blocks of 256: more than a grid's second dimension holds."""
    import cnn_convolution_implicit_gb300 as cg
    C = 256 * 65535 + 1
    g = torch.Generator().manual_seed(5)
    x, dy = torch.randn(1, 1, 1, C, generator=g), torch.randn(1, 1, 1, C, generator=g)
    gamma, beta = torch.randn(C, generator=g) * 0.3 + 1.0, torch.randn(C, generator=g) * 0.3
    stats = torch.empty(2, 1, 1, device="cuda")
    y = cg.group_norm(x.cuda(), 1, gamma.cuda(), beta.cuda(), act="silu", stats=stats)
    want, tol = ref.norm_forward(_flat(x), 1, _np(gamma), _np(beta), 1e-5, "silu")
    ref.check(_flat(y), want, tol, False, "y")
    got = cg.group_norm_backward(dy.cuda(), x.cuda(), stats, 1, gamma.cuda(), beta.cuda(), act="silu")
    want, tol = ref.norm_backward(_flat(dy), _flat(x), stats.cpu().numpy(), 1, _np(gamma), _np(beta), "silu")
    for a, b, t, name in zip((_flat(got[0]), _np(got[1]), _np(got[2])), want, tol, ("dx", "dgamma", "dbeta")):
        ref.check(a, b, t, False, name)


@pytest.mark.parametrize("shape,dtype", [((1 << 19, 1, 1, 32, 4), "f32"), ((1 << 18, 1, 1, 21, 3), "f32"),
                                         ((1 << 17, 2, 2, 64, 8), "bf16")])
def test_affine_gradients_of_many_images(shape, dtype):
    """Rows of tokens, each an image: dgamma and dbeta add up hundreds of thousands of partial sums
    of one sign, whose rounding must not pile up."""
    import cnn_convolution_implicit_gb300 as cg
    N, H, W, C, G = shape
    x, gamma, beta = _make(N, H, W, C, dtype, 23)
    dy = torch.full(x.shape, 0.1).to(DT[dtype])
    stats = torch.empty(2, N, G, device="cuda")
    cg.group_norm(x.cuda(), G, gamma.cuda(), beta.cuda(), stats=stats)
    got = cg.group_norm_backward(dy.cuda(), x.cuda(), stats, G, gamma.cuda(), beta.cuda())
    want, tol = ref.norm_backward(_flat(dy), _flat(x), stats.cpu().numpy(), G, _np(gamma), _np(beta), "none")
    ref.check(_np(got[1]), want[1], tol[1], False, "dgamma")
    ref.check(_np(got[2]), want[2], tol[2], False, "dbeta")


@pytest.mark.parametrize("act", ["none", "silu"])
def test_a_plan_is_the_same_after_other_calls(act):
    """The form of a plan comes from its shape and the device, not from the maps that went before:
    small ones must not leave the kernels less shared memory than a larger one counts on."""
    import cnn_convolution_implicit_gb300 as cg
    large = [(64, 256, 56, 56, 32), (8, 64, 56, 56, 16), (20, 512, 14, 14, 32)]
    small = [(4, 64, 56, 56, 32), (2, 128, 16, 16, 16), (1, 256, 8, 8, 32)]
    for dtype in ("bf16", "f32"):
        made = [cg.GroupNormPlan(N, C, H, W, G, dtype, act=act).workspace_bytes for N, C, H, W, G in large]
        for N, C, H, W, G in small:
            plan = cg.GroupNormPlan(N, C, H, W, G, dtype, act=act)
            x, stats = torch.randn(plan.shape, device="cuda").to(DT[dtype]), plan.empty_stats()
            plan.forward(x, stats=stats)
            plan.forward_int8(x)
            plan.backward(x, x, stats)
        again = [cg.GroupNormPlan(N, C, H, W, G, dtype, act=act).workspace_bytes for N, C, H, W, G in large]
        assert again == made
    torch.cuda.synchronize()


def test_silu_over_its_range():
    """SiLU in FP32, of the norm (flat groups give act(beta)), of its gradient and of the product (no
    sum: act(bias)).  exp(-z) is 2^(-z log2 e): the product's rounding and the constant's are 1.5 * 2^-24
    |z| of it, the approximate power 4 * 2^-24, the reciprocal and the sums about it another 4; and
    1 - sigmoid loses as much again where it cancels."""
    import cnn_convolution_implicit_gb300 as cg
    z = torch.linspace(-85.0, 85.0, 4096)
    y = cg.group_norm(torch.ones(1, 2, 2, 4096, device="cuda"), 32, None, z.cuda(), act="silu")
    want = ref.activation(_np(z), "silu")
    bound = (1.5 * np.abs(_np(z)) + 8.0) * ref.U32
    assert np.all(np.abs(_np(y)[0, 0, 0] - want) <= bound * np.abs(want))
    for rows in (1, 16, 128):  # the kernels of few rows, of 5 to 64, of many
        p = cg.int8_matmul(torch.zeros(rows, 16, dtype=torch.int8, device="cuda"), torch.ones(rows, device="cuda"),
                           torch.ones(4096, 16, dtype=torch.int8, device="cuda"), torch.ones(4096, device="cuda"), z.cuda(),
                           act="silu", out="f32")
        assert np.all(np.abs(_np(p)[-1] - want) <= bound * np.abs(want))
    stats = torch.tensor([[[0.0]], [[1.0]]]).repeat(1, 1, 32).cuda()
    _, _, dbeta = cg.group_norm_backward(torch.ones(1, 1, 1, 4096, device="cuda"), torch.zeros(1, 1, 1, 4096, device="cuda"),
                                         stats, 32, None, z.cuda(), act="silu")
    s = 1.0 / (1.0 + np.exp(-_np(z)))
    grad, size = s * (1.0 + _np(z) * (1.0 - s)), s * (1.0 + np.abs(_np(z)))
    assert np.all(np.abs(_np(dbeta) - grad) <= 2 * bound * size)
