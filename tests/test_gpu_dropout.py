"""Dropout on the GPU against the published generator restated in 64-bit integers: the mask element by
element, both types, odd lengths, residuals, aliases, p from 0 to 1, counters past 32 bits of
elements, graphs whose state moves, autograd."""
import numpy as np
import pytest
import torch

import operator_refs as oref
import row_refs as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.detach().double().cpu().numpy()


def _state(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 15, 17, 1000, 4099, 301 * 777, 1 << 20, (1 << 22) + 5])
def test_mask_and_values(n, dtype):
    import cnn_convolution_implicit_gb300 as cg
    g = torch.Generator().manual_seed(n)
    x, r = (torch.randn(n, generator=g).to(DTYPES[dtype]) for _ in range(2))
    x[x == 0] = 1.0
    seed, offset, p = 0x123456789ABCDEF + n, (5 << 32) + n, 0.25
    state = _state(seed, offset).cuda()
    keep = ref.dropout_keep(seed, offset, p, 0, n)
    canvas = torch.full((n + 64,), 7.0, device="cuda", dtype=DTYPES[dtype])
    y = cg.dropout(x.cuda(), p, state, y=canvas[:n])
    assert np.array_equal(_np(y) != 0, keep) and torch.all(canvas[n:] == 7.0)
    want, tol = ref.dropout(_np(x), None, keep, p)
    oref.check(_np(y), want, tol, dtype == "bf16", "y")
    want, tol = ref.dropout(_np(x), _np(r), keep, p)
    oref.check(_np(cg.dropout(x.cuda(), p, state, residual=r.cuda())), want, tol, dtype == "bf16", "y with residual")
    assert torch.equal(cg.dropout_backward(x.cuda(), p, state), y)


@pytest.mark.parametrize("p", [0.0, 1e-9, 2.0 ** -32, 0.5, 0.999, 1.0 - 2.0 ** -40, 1.0])
def test_probabilities(p):
    import cnn_convolution_implicit_gb300 as cg
    n = 100003
    x = torch.randn(n, generator=torch.Generator().manual_seed(1)).abs() + 0.5
    y = cg.dropout(x.cuda(), p, _state(-1, -2).cuda())     # all 64 bits of the state count
    keep = ref.dropout_keep((1 << 64) - 1, (1 << 64) - 2, p, 0, n)
    assert np.array_equal(_np(y) != 0, keep)
    if p in (0.0, 1.0):
        assert torch.equal(y.cpu(), x * (1.0 - p))
    want, tol = ref.dropout(_np(x), None, keep, p)
    oref.check(_np(y), want, tol, False, "y")
    share = float(keep.mean())
    assert abs(share - (1 - p)) <= 6 * (p * (1 - p) / n) ** 0.5 + 1e-6


def test_bad_values_in_dropped_places():
    import cnn_convolution_implicit_gb300 as cg
    n = 4096
    keep = ref.dropout_keep(3, 4, 0.5, 0, n)
    x = torch.ones(n)
    x[torch.from_numpy(~keep)] = torch.tensor([float("nan"), float("inf")]).repeat(n)[:int((~keep).sum())]
    y = cg.dropout(x.cuda(), 0.5, _state(3, 4).cuda())
    assert np.array_equal(_np(y), np.where(keep, 2.0, 0.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_buffers_that_are_inputs(dtype):
    import cnn_convolution_implicit_gb300 as cg
    x, r = (torch.randn(1003, device="cuda").to(DTYPES[dtype]) for _ in range(2))
    state = _state(8, 9).cuda()
    y = cg.dropout(x, 0.3, state, residual=r)
    x2, r2 = x.clone(), r.clone()
    assert torch.equal(cg.dropout(x2, 0.3, state, residual=r, y=x2), y)
    assert torch.equal(cg.dropout(x, 0.3, state, residual=r2, y=r2), y)


def test_past_2_32_elements():
    import cnn_convolution_implicit_gb300 as cg
    n = (1 << 32) + 21
    x = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    y = cg.dropout(x, 0.5, _state(11, 12).cuda(), y=x)
    for first in (0, (1 << 31) - 16, (1 << 32) - 16, n - 21):
        keep = ref.dropout_keep(11, 12, 0.5, first, 21)
        assert np.array_equal(_np(y[first:first + 21]), np.where(keep, 2.0, 0.0))


def test_graph_takes_the_state_of_each_replay():
    import cnn_convolution_implicit_gb300 as cg
    x, state = torch.ones(5000, device="cuda"), _state(1, 0).cuda()
    graph = torch.cuda.CUDAGraph()
    cg.dropout(x, 0.4, state)
    with torch.cuda.graph(graph):
        y = cg.dropout(x, 0.4, state)
        state[1] += 1
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(_np(y) != 0, ref.dropout_keep(1, step, 0.4, 0, 5000))
    side = torch.cuda.Stream()
    state.copy_(_state(1, 2))
    side.wait_stream(torch.cuda.current_stream())
    z = cg.dropout(x, 0.4, state, stream=side)
    side.synchronize()
    assert torch.equal(y, z)


def test_gradients_are_recorded():
    """The backward pass draws the mask of its own forward pass, whatever became of the state since."""
    import cnn_convolution_implicit_gb300 as cg
    x, r = (torch.randn(7, 33, device="cuda", requires_grad=True) for _ in range(2))
    state = _state(21, 22).cuda()
    y = cg.dropout(x, 0.25, state, residual=r)
    state += 5
    dy = torch.randn(7, 33, device="cuda")
    y.backward(dy)
    keep = ref.dropout_keep(21, 22, 0.25, 0, 7 * 33).reshape(7, 33)
    want, tol = ref.dropout(_np(dy), None, keep, 0.25)
    oref.check(_np(x.grad), want, tol, False, "dx")
    assert torch.equal(r.grad, dy)
    with pytest.raises(ValueError):
        cg.dropout(x, 0.25, state, y=torch.empty_like(x))
    # linear in x: a difference is exact up to its own rounding
    with torch.no_grad():
        a, b = cg.dropout(x, 0.25, state), cg.dropout(x + 1, 0.25, state)
    keep = ref.dropout_keep(26, 27, 0.25, 0, 7 * 33).reshape(7, 33)
    assert np.allclose(_np(b - a), keep / 0.75, rtol=0, atol=4e-6)


def test_refusals():
    import cnn_convolution_implicit_gb300 as cg
    x, state = torch.ones(4, 64, device="cuda"), _state(1, 2).cuda()
    for bad in (dict(x=x.cpu()), dict(x=x.half()), dict(x=x.t()), dict(state=state.cpu()), dict(state=state.int()),
                dict(state=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(residual=x[:2]), dict(residual=x.bfloat16()),
                dict(y=x.bfloat16())):
        with pytest.raises(ValueError):
            cg.dropout(**dict(dict(x=x, p=0.1, state=state), **bad))
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(cg.ConvError):
            cg.dropout(x, p, state)
    with pytest.raises(cg.ConvError):
        cg.dropout(x[:0], 0.1, state)
