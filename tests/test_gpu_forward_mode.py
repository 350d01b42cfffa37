"""Forward-mode derivatives: no operator carries a tangent, and a tensor that has one is refused, in the
functional forms and in the backward passes that they record, instead of losing it without a word."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _tensors():
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *shape: torch.randn(*shape, device="cuda", generator=g)
    return {"x": new(6, 16).to(BF16), "w": new(8, 16).to(BF16), "bias": new(8), "residual": new(6, 8).to(BF16), "z": new(6, 8).to(BF16),
            "dy": new(6, 8).to(BF16), "gamma": new(16), "stream": new(6, 16).to(BF16), "rstd": new(6).abs(),
            "map": new(2, 4, 4, 16), "beta": new(16), "stats": new(2, 2, 4).abs(), "state": torch.tensor([3, 4], device="cuda")}


CALLS = {
    "linear": (lambda cg, t: cg.linear(t["x"], t["w"], t["bias"], "silu", t["residual"]), ("x", "w", "bias", "residual")),
    "linear_backward": (lambda cg, t: cg.linear_backward(t["dy"], t["x"], t["w"], t["z"], "silu"), ("dy", "x", "w", "z")),
    "rms_norm": (lambda cg, t: cg.rms_norm(t["x"], t["gamma"], t["stream"]), ("x", "gamma", "stream")),
    "rms_norm_backward": (lambda cg, t: cg.rms_norm_backward(t["x"], t["stream"], t["rstd"], t["gamma"], t["x"]),
                          ("x", "stream", "rstd", "gamma")),
    "dropout": (lambda cg, t: cg.dropout(t["x"], 0.3, t["state"], t["stream"]), ("x", "stream")),
    "dropout_backward": (lambda cg, t: cg.dropout_backward(t["x"], 0.3, t["state"]), ("x",)),
    "group_norm": (lambda cg, t: cg.group_norm(t["map"], 4, t["gamma"], t["beta"]), ("map", "gamma", "beta")),
    "group_norm_backward": (lambda cg, t: cg.group_norm_backward(t["map"], t["map"], t["stats"], 4, t["gamma"], t["beta"]),
                            ("map", "stats", "gamma", "beta")),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tangents_are_refused(name):
    import cnn_convolution_implicit_gb300 as cg
    call, inputs = CALLS[name]
    t = _tensors()
    first = call(cg, t)
    first = first if isinstance(first, tuple) else (first,)
    for which in inputs:
        with fwad.dual_level():
            dual = dict(t, **{which: fwad.make_dual(t[which], torch.ones_like(t[which]))})
            with pytest.raises(ValueError, match="forward-mode"):
                call(cg, dual)
            with torch.no_grad(), pytest.raises(ValueError, match="forward-mode"):
                call(cg, dual)
            again = call(cg, t)  # tensors without a tangent go as ever, inside the level too
            again = again if isinstance(again, tuple) else (again,)
            assert all(torch.equal(p, q) for p, q in zip(first, again))
        call(cg, t)


@pytest.mark.parametrize("name", ["linear", "rms_norm", "dropout", "group_norm"])
def test_tangents_of_upstream_gradients_are_refused(name):
    """Forward over reverse: the gradient that reaches a recorded backward pass has a tangent."""
    import cnn_convolution_implicit_gb300 as cg
    call, inputs = CALLS[name]
    t = _tensors()
    t[inputs[0]].requires_grad_(True)
    out = call(cg, t)
    out = out[0] if isinstance(out, tuple) else out
    with fwad.dual_level():
        up = fwad.make_dual(torch.ones_like(out), torch.ones_like(out))
        with pytest.raises(ValueError, match="forward-mode"):
            torch.autograd.grad(out, t[inputs[0]], up)


def test_function_transforms_are_refused():
    import cnn_convolution_implicit_gb300 as cg
    t = _tensors()
    one = torch.ones_like(t["x"])
    for call in (lambda x: cg.linear(x, t["w"]), lambda x: cg.rms_norm(x), lambda x: cg.dropout(x, 0.1, t["state"])):
        with pytest.raises((ValueError, RuntimeError)):
            torch.func.jvp(call, (t["x"],), (one,))
