"""Tensors on another device than the current one are refused before anything is planned or
launched (host-side, with stand-ins for tensors of a second device): a plan belongs to the device
that was current when it was made, and a launch goes to the current one."""
import pytest
import torch

import cnn_convolution_implicit_gb300 as cg
from cnn_convolution_implicit_gb300 import binding, operators


class OnDevice:
    """A contiguous tensor's surface, on CUDA device ``index``."""
    is_cuda = True

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        raise AssertionError("a pointer of another device was taken")


@pytest.fixture
def current(monkeypatch):
    """Device 0 is current; nothing may reach the library's calls."""
    operators._torch()
    monkeypatch.setattr(operators, "_current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)  # as the convolutions ask
    for cache in (operators._norm_plans, operators._int8_plans, binding._plan_cache):
        cache.clear()
    yield
    assert not operators._norm_plans and not operators._int8_plans and not binding._plan_cache


BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def _calls(index):
    x4, rows = OnDevice((1, 4, 4, 32), BF16, index), OnDevice((4, 16), BF16, index)
    q, w = OnDevice((4, 16), I8, index), OnDevice((8, 16), I8, index)
    v4, v8 = OnDevice((4,), F32, index), OnDevice((8,), F32, index)
    stats = OnDevice((2, 1, 4), F32, index)
    return {
        "group_norm": lambda: cg.group_norm(x4, 4),
        "group_norm_int8": lambda: cg.group_norm_int8(x4, 4),
        "group_norm_backward": lambda: cg.group_norm_backward(x4, x4, stats, 4),
        "int8_matmul": lambda: cg.int8_matmul(q, v4, w, v8),
        "int8_linear": lambda: cg.int8_linear(rows, w, v8),
        "quantize_rows": lambda: cg.quantize_rows(rows),
        "conv2d": lambda: cg.conv2d(x4, OnDevice((8, 3, 3, 32), BF16, index)),
        "GroupNormPlan.forward": lambda: cg.GroupNormPlan(1, 32, 4, 4, 4).forward(x4),
        "GroupNormPlan.backward": lambda: cg.GroupNormPlan(1, 32, 4, 4, 4).backward(x4, x4, stats),
        "Int8MatmulPlan.forward": lambda: cg.Int8MatmulPlan(4, 8, 16).forward(q, v4, w, v8),
        "Int8MatmulPlan.forward_quantize": lambda: cg.Int8MatmulPlan(4, 8, 16).forward_quantize(rows, w, v8),
        "ConvPlan.forward": lambda: cg.ConvPlan(1, 32, 4, 4, 8, 3, 3, bias=False).forward(x4, OnDevice((8, 3, 3, 32), BF16, index)),
        "BlockPlan.forward": lambda: cg.BlockPlan(1, 64, 8, 8, 64).forward(
            OnDevice((1, 8, 8, 64), F32, index), OnDevice((64, 3, 3), F32, index), OnDevice((64, 64), BF16, index)),
    }


@pytest.mark.parametrize("name", sorted(_calls(1)))
def test_tensors_of_another_device_are_refused(name, current):
    with pytest.raises(ValueError, match="cuda:0 is current"):
        _calls(1)[name]()


def test_mixed_devices_are_refused(current):
    x, w = OnDevice((1, 4, 4, 32), BF16, 0), OnDevice((8, 3, 3, 32), BF16, 0)
    plan = cg.ConvPlan(1, 32, 4, 4, 8, 3, 3, P=1, bias=True)
    bias = OnDevice((8,), F32, 0)
    for swap in ("w", "bias", "y", "scale"):
        args = {"w": w, "bias": bias, "y": None, "scale": None}
        args[swap] = OnDevice(*{"w": ((8, 3, 3, 32), BF16), "bias": ((8,), F32), "y": ((1, 4, 4, 8), BF16),
                                "scale": ((8,), F32)}[swap], 1)
        with pytest.raises(ValueError, match="one device"):
            plan.forward(x, **args)
    with pytest.raises(ValueError, match="one device"):
        plan.forward(x, w, bias, y=torch.empty(1, 4, 4, 8, dtype=BF16))     # host memory
    with pytest.raises(ValueError):
        cg.GroupNormPlan(1, 32, 4, 4, 4).forward(x, OnDevice((32,), F32, 1))
    with pytest.raises(ValueError):
        cg.BlockPlan(1, 64, 8, 8, 64).forward(OnDevice((1, 8, 8, 64), F32, 0), OnDevice((64, 3, 3), F32, 1),
                                              OnDevice((64, 64), BF16, 0))
