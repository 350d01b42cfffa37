"""What a recorded call keeps and what its backward pass reads: a gradient that nobody gave is not made up of zeros, and no
tensor stays alive that no wanted gradient reads."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _norm(dtype, M=10, C=96):
    g = torch.Generator(device="cuda").manual_seed(5)
    x, r, dy = (torch.randn(M, C, device="cuda", generator=g).to(dtype) for _ in range(3))
    return x, r, dy, torch.randn(C, device="cuda", generator=g)


@pytest.fixture
def upstream(monkeypatch):
    """The dh of every backward pass of the norm."""
    import cnn_convolution_implicit_gb300 as cg
    seen, plain = [], cg.RmsNormPlan.backward

    def backward(self, dy, h, rstd, gamma=None, dh=None, *more, **named):
        seen.append(dh)
        return plain(self, dy, h, rstd, gamma, dh, *more, **named)

    monkeypatch.setattr(cg.RmsNormPlan, "backward", backward)
    return seen


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_an_h_that_nobody_uses(dtype, upstream):
    import cnn_convolution_implicit_gb300 as cg
    x, r, dy, gamma = _norm(dtype)
    rstd = torch.empty(10, device="cuda")
    _, h = cg.rms_norm(x, gamma, r, rstd=rstd)
    want = cg.rms_norm_backward(dy, h, rstd, gamma)
    upstream.clear()
    leaves = [t.clone().requires_grad_(True) for t in (x, r, gamma)]
    y, _ = cg.rms_norm(leaves[0], leaves[2], leaves[1])
    y.backward(dy)
    assert len(upstream) == 1 and upstream[0] is None
    assert torch.equal(leaves[0].grad, want[0]) and torch.equal(leaves[1].grad, want[0]) and torch.equal(leaves[2].grad, want[1])


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_a_y_that_nobody_uses(dtype, upstream):
    """dx is dh, dgamma zero."""
    import cnn_convolution_implicit_gb300 as cg
    x, r, dh, gamma = _norm(dtype)
    leaves = [t.clone().requires_grad_(True) for t in (x, r, gamma)]
    _, h = cg.rms_norm(leaves[0], leaves[2], leaves[1])
    h.backward(dh)
    assert not upstream
    assert torch.equal(leaves[0].grad, dh) and torch.equal(leaves[1].grad, dh)
    assert torch.equal(leaves[2].grad, torch.zeros_like(gamma))
    # gamma or x alone, a gradient that is not contiguous, and gradients that autograd adds up
    for wanted in ("gamma", "x"):
        one = (gamma if wanted == "gamma" else x).clone().requires_grad_(True)
        _, h = cg.rms_norm(one if wanted == "x" else x, one if wanted == "gamma" else gamma, r)
        wide = torch.zeros(10, 192, device="cuda", dtype=dtype)
        wide[:, ::2] = dh
        h.backward(wide[:, ::2])
        assert torch.equal(one.grad, dh if wanted == "x" else torch.zeros_like(gamma))
    both = x.clone().requires_grad_(True)
    _, h = cg.rms_norm(both, gamma, both)
    h.backward(dh)
    assert torch.equal(both.grad, dh + dh)


def test_both_outputs_used(upstream):
    import cnn_convolution_implicit_gb300 as cg
    x, r, dy, gamma = _norm(BF16)
    rstd = torch.empty(10, device="cuda")
    _, h0 = cg.rms_norm(x, gamma, r, rstd=rstd)
    want = cg.rms_norm_backward(dy, h0, rstd, gamma, r)
    leaf = x.clone().requires_grad_(True)
    y, h = cg.rms_norm(leaf, gamma, r)
    torch.autograd.backward([y, h], [dy, r])
    assert torch.equal(leaf.grad, want[0])


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("wanted", ["x", "w", "bias", "residual"])
def test_linear_keeps_what_its_gradients_read(act, wanted):
    import cnn_convolution_implicit_gb300 as cg
    g = torch.Generator(device="cuda").manual_seed(6)
    t = {"x": torch.randn(12, 40, device="cuda", generator=g).to(BF16), "w": torch.randn(24, 40, device="cuda", generator=g).to(BF16),
         "bias": torch.randn(24, device="cuda", generator=g), "residual": torch.randn(12, 24, device="cuda", generator=g).to(BF16)}
    dy, z = torch.randn(12, 24, device="cuda", generator=g).to(BF16), torch.empty(12, 24, device="cuda", dtype=BF16)
    cg.linear(t["x"], t["w"], t["bias"], act, t["residual"], z=z)
    want = dict(zip(("x", "w", "bias"), cg.linear_backward(dy, t["x"], t["w"], z, act)), residual=dy)
    t[wanted].requires_grad_(True)
    y = cg.linear(t["x"], t["w"], t["bias"], act, t["residual"])
    x, w, z = y.grad_fn.saved_tensors
    assert (x is not None) == (wanted == "w") and (w is not None) == (wanted == "x")
    assert (z is not None) == (act != "none" and wanted != "residual")
    y.backward(dy)
    assert torch.equal(t[wanted].grad, want[wanted])
