"""A quantised bottleneck and its normalisation's training step, on the library's kernels:

    3x3 convolution -> group norm + SiLU -> 8-bit pixels -> pointwise (1x1) product in 8 bits

The pointwise layer's weights are brought to 8 bits once (one scale per output channel); the
pixels are brought to 8 bits by the norm itself (one scale per pixel), so the product reads a
quarter of what FP32 pixels would take.  The second part runs the norm as training does:
forward with its statistics, then the gradients of its input, gamma and beta.

    python examples/quantized_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import cnn_convolution_implicit_gb300 as cg  # noqa: E402


def main(N=4, C_in=128, H=56, W=56, C=256, C_out=512, groups=32):
    g = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape, std=1.0):
        return torch.randn(shape, device="cuda", generator=g) * std

    x = randn(N, H, W, C_in).to(torch.bfloat16)
    w3 = randn(C, 3, 3, C_in, std=(2.0 / (9 * C_in)) ** 0.5).to(torch.bfloat16)
    gamma, beta = 1.0 + randn(C, std=0.1), randn(C, std=0.1)
    w1, b1 = randn(C_out, C, std=C ** -0.5), randn(C_out, std=0.1)
    w1_q, w1_scale = cg.quantize_rows(w1)  # once, as a deployment would

    conv = cg.conv2d(x, w3, padding=1)
    q, scale = cg.group_norm_int8(conv, groups, gamma, beta, act="silu")
    y = cg.int8_matmul(q, scale, w1_q, w1_scale, b1)

    # the same without 8 bits, in FP32
    h = conv.float().view(N, -1, groups, C // groups)
    h = (h - h.mean((1, 3), keepdim=True)) * (h.var((1, 3), unbiased=False, keepdim=True) + 1e-5).rsqrt()
    h = torch.nn.functional.silu(h.reshape(N, H, W, C) * gamma + beta)
    want = h @ w1.t() + b1
    err = float((y.float() - want).norm() / want.norm())
    print("block [%d,%d,%d,%d] -> %s, 8-bit error against FP32 %.2f %%" % (N, H, W, C_in, list(y.shape), 100 * err))

    # a training step of the norm: gradients of 0.5 * |out|^2
    plan = cg.GroupNormPlan(N, C, H, W, groups, "bf16", act="silu")
    stats = plan.empty_stats()
    out = plan.forward(conv, gamma, beta, stats=stats)
    dx, dgamma, dbeta = plan.backward(out, conv, stats, gamma, beta)
    print("norm's gradients: |dx| %.3e  |dgamma| %.3e  |dbeta| %.3e"
          % tuple(float(t.float().norm()) for t in (dx, dgamma, dbeta)))
    torch.cuda.synchronize()
    assert cg.device_status() == 0
    return err


if __name__ == "__main__":
    main()
