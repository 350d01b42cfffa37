"""Buffers that a call is given for its results: autograd learns that they were written, so a backward pass that
saved one refuses instead of reading what came later."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _cases(cg):
    """name: (shape and type of the buffer, call that writes it)"""
    x, w = torch.ones(6, 16, device="cuda", dtype=BF16), torch.ones(16, 16, device="cuda", dtype=BF16)
    f, rows = torch.ones(16, device="cuda"), torch.ones(6, device="cuda")
    state = torch.tensor([3, 4], device="cuda")
    linear, norm = cg.LinearPlan(6, 16, 16, "relu"), cg.RmsNormPlan(6, 16)
    image = torch.ones(2, 3, 3, 16, device="cuda")
    product, conv = cg.Int8MatmulPlan(6, 16, 16), cg.ConvPlan(2, 8, 4, 4, 8, 1, 1, 1, 0, 1, 1, "f32", bias=False)
    q, weights, scale = torch.ones(6, 16, device="cuda", dtype=torch.int8), torch.ones(16, 16, device="cuda", dtype=torch.int8), f
    pixels, taps = torch.ones(2, 4, 4, 8, device="cuda"), torch.ones(8, 1, 1, 8, device="cuda")
    block = cg.BlockPlan(1, 64, 8, 8, 64)
    branch = (torch.ones(1, 8, 8, 64, device="cuda"), torch.ones(64, 3, 3, device="cuda"), torch.ones(64, 64, device="cuda", dtype=BF16))
    return {
        "linear y": (x, lambda b: cg.linear(x, w, y=b)), "linear y over the residual": (x, lambda b: cg.linear(x, w, residual=b, y=b)),
        "linear z": (x, lambda b: cg.linear(x, w, act="relu", z=b)),
        "LinearPlan y": (x, lambda b: linear.forward(x, w, y=b)), "LinearPlan z": (x, lambda b: linear.forward(x, w, z=b)),
        "LinearPlan dx": (x, lambda b: linear.backward(x, x, w, x, dx=b)), "LinearPlan dw": (w, lambda b: linear.backward(x, x, w, x, dw=b)),
        "LinearPlan dbias": (f, lambda b: linear.backward(x, x, w, x, dbias=b)),
        "rms_norm h over the residual": (x, lambda b: cg.rms_norm(x, residual=b, h=b)), "rms_norm rstd": (rows, lambda b: cg.rms_norm(x, rstd=b)),
        "rms_norm_int8 h": (x, lambda b: cg.rms_norm_int8(x, residual=x, h=b)), "rms_norm_int8 rstd": (rows, lambda b: cg.rms_norm_int8(x, rstd=b)),
        "RmsNormPlan y": (x, lambda b: norm.forward(x, y=b)), "RmsNormPlan scale": (rows, lambda b: norm.forward_int8(x, scale=b)),
        "RmsNormPlan dx over dy": (x, lambda b: norm.backward(b, x, rows, dx=b)), "RmsNormPlan dgamma": (f, lambda b: norm.backward(x, x, rows, dgamma=b)),
        "dropout y": (x, lambda b: cg.dropout(x, 0.5, state, y=b)), "dropout y over x": (x, lambda b: cg.dropout(b, 0.5, state, y=b)),
        "group_norm y": (image, lambda b: cg.group_norm(image, 4, y=b)),
        "int8 y": (x, lambda b: product.forward(q, rows, weights, scale, y=b)), "quantised y": (x, lambda b: product.forward_quantize(x, weights, scale, y=b)),
        "convolution y": (torch.ones(2, 4, 4, 8, device="cuda"), lambda b: conv.forward(pixels, taps, y=b)),
        "block y": (torch.ones(1, 8, 8, 64, device="cuda", dtype=BF16), lambda b: block.forward(*branch, y=b)),
        "group_norm stats": (torch.ones(2, 2, 4, device="cuda"), lambda b: cg.group_norm(image, 4, stats=b)),
    }


NAMES = ["linear y", "linear y over the residual", "linear z", "LinearPlan y", "LinearPlan z", "LinearPlan dx", "LinearPlan dw", "LinearPlan dbias",
         "rms_norm h over the residual", "rms_norm rstd", "rms_norm_int8 h", "rms_norm_int8 rstd", "RmsNormPlan y", "RmsNormPlan scale",
         "RmsNormPlan dx over dy", "RmsNormPlan dgamma", "dropout y", "dropout y over x", "group_norm y", "group_norm stats", "int8 y", "quantised y", "convolution y", "block y"]


@pytest.mark.parametrize("name", NAMES)
def test_a_saved_buffer_that_was_written_is_noticed(name):
    import cnn_convolution_implicit_gb300 as cg
    like, call = _cases(cg)[name]
    buffer = like.clone()
    leaf = torch.full_like(buffer, 2.0, requires_grad=True)
    y = leaf * buffer                     # saves the buffer for the leaf's gradient
    call(buffer)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_every_buffer_is_covered():
    import cnn_convolution_implicit_gb300 as cg
    assert sorted(_cases(cg)) == sorted(NAMES)


@pytest.mark.parametrize("name", NAMES)
def test_in_inference_mode(name):
    """Tensors made in inference mode keep no versions; the calls take them there."""
    import cnn_convolution_implicit_gb300 as cg
    with torch.inference_mode():
        like, call = _cases(cg)[name]
        call(like.clone())


def test_a_buffer_of_inference_mode_outside_of_it():
    import cnn_convolution_implicit_gb300 as cg
    with torch.inference_mode():
        like, _ = _cases(cg)["linear y"]
        buffer = like.clone()
    _, call = _cases(cg)["linear y"]
    call(buffer)
    assert torch.all(buffer == 16)
