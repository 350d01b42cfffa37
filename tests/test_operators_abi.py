"""Host-side checks of the group norm and 8-bit product calls (no GPU needed): shapes, flags
and pointers are refused with their status before anything is launched."""
import ctypes

import pytest
import torch

import cnn_convolution_implicit_gb300 as cg

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("args,status", [
    ((0, 32, 4, 4, 4, 1e-5, 1, 0), 1),
    ((1, 0, 4, 4, 4, 1e-5, 1, 0), 1),
    ((1, 32, 0, 4, 4, 1e-5, 1, 0), 1),
    ((1, 32, 4, -1, 4, 1e-5, 1, 0), 1),
    ((1, 32, 4, 4, 0, 1e-5, 1, 0), 1),
    ((1, 32, 4, 4, 5, 1e-5, 1, 0), 1),       # C % groups
    ((1, 32, 4, 4, 4, -1e-5, 1, 0), 1),
    ((1, 32, 4, 4, 4, NAN, 1, 0), 1),
    ((1, 32, 4, 4, 4, INF, 1, 0), 1),
    ((1, 32, 4, 4, 4, 1e-5, 2, 0), 1),       # dtype
    ((1, 32, 4, 4, 4, 1e-5, 1, 3), 1),       # act
    ((1, 32, 1 << 16, 1 << 15, 4, 1e-5, 1, 0), 2),   # 2^31 pixels
    ((1 << 20, 32, 1, 1, 32, 1e-5, 1, 0), 2),        # 2^25 (image, group) pairs
    ((1, 32, 4, 4, 4, 0.0, 1, 2), 0),
    ((1, 7, 3, 5, 7, 1e-5, 0, 1), 0),
])
def test_group_norm_create(args, status):
    L = cg.lib()
    h = ctypes.c_void_p(1234)
    assert L.conv_group_norm_plan_create(ctypes.byref(h), *args) == status
    assert (h.value is None) == (status != 0)
    if h.value:
        assert L.conv_group_norm_plan_destroy(h) == 0


@pytest.mark.parametrize("args,status", [
    ((0, 8, 8, 1, 0), 1), ((8, 0, 8, 1, 0), 1), ((8, 8, -1, 1, 0), 1), ((8, 8, 8, 5, 0), 1), ((8, 8, 8, 1, 9), 1),
    ((8, 8, 131072, 1, 0), 2), ((1 << 30, 8, 2048, 1, 0), 2), ((1 << 30, 1 << 20, 8, 1, 0), 2),
    ((1, 1, 131071, 0, 2), 0), ((1, 1, 1, 1, 1), 0),
])
def test_int8_create(args, status):
    L = cg.lib()
    h = ctypes.c_void_p(1234)
    assert L.conv_int8_plan_create(ctypes.byref(h), *args) == status
    assert (h.value is None) == (status != 0)
    if h.value:
        assert L.conv_int8_plan_destroy(h) == 0


def test_null_and_misaligned_pointers():
    L = cg.lib()
    assert L.conv_group_norm_plan_create(None, 1, 32, 4, 4, 4, 1e-5, 1, 0) == 1
    assert L.conv_int8_plan_create(None, 1, 8, 8, 1, 0) == 1
    assert L.conv_group_norm_plan_destroy(None) == 0 and L.conv_int8_plan_destroy(None) == 0
    assert L.conv_group_norm_workspace(None, None, None, None) == 1 and L.conv_int8_workspace(None, None, None) == 1
    assert L.conv_int8_plan_device_status(None, None, None) == 1
    n = cg.GroupNormPlan(1, 32, 4, 4, 4)
    A = 256
    fwd, q8, bwd = L.conv_group_norm_forward, L.conv_group_norm_forward_int8, L.conv_group_norm_backward
    assert fwd(None, A, None, None, A, None, A, None) == 1
    assert fwd(n._plan, None, None, None, A, None, A, None) == 1
    assert fwd(n._plan, A, None, None, None, None, A, None) == 1
    wide = cg.GroupNormPlan(1, 7, 4, 4, 7)     # odd channels: sums by channel, in a workspace
    assert wide.workspace_bytes["forward"] > 0 and fwd(wide._plan, A, None, None, A, None, None, None) == 1
    assert fwd(n._plan, A + 2, None, None, A, None, A, None) == 3
    assert fwd(n._plan, A, A + 4, None, A, None, A, None) == 3
    assert fwd(n._plan, A, None, None, A, A + 8, A, None) == 3
    assert q8(n._plan, A, None, None, A, None, None, A, None) == 1
    assert q8(n._plan, A, None, None, A + 1, A, None, A, None) == 3
    assert bwd(n._plan, A, A, None, None, None, A, A, A, A, None) == 1          # no stats
    assert bwd(n._plan, A, A, A, None, None, A, A, None, A, None) == 1          # dgamma without dbeta
    assert bwd(n._plan, A, A, A, None, None, A + 8, A, A, A, None) == 3
    p = cg.Int8MatmulPlan(4, 8, 16)
    f, g = L.conv_int8_forward, L.conv_int8_forward_quantize
    assert f(None, A, A, A, A, None, A, A, None) == 1
    assert f(p._plan, A, None, A, A, None, A, A, None) == 1
    assert f(p._plan, A, A, A, A, None, None, A, None) == 1
    assert f(p._plan, A + 1, A, A, A, None, A, A, None) == 3
    assert f(p._plan, A, A, A, A, A + 4, A, A, None) == 3
    assert f(p._plan, A, A, A, A, None, A, A + 8, None) == 3
    odd = cg.Int8MatmulPlan(400, 8, 20)
    assert odd.workspace_bytes["forward"] > 0 and f(odd._plan, A, A, A, A, None, A, None, None) == 1  # rows to lay out
    assert g(p._plan, None, 1, A, A, None, A, A, None) == 1
    assert g(p._plan, A, 7, A, A, None, A, A, None) == 1
    assert p.workspace_bytes == {"forward": 0, "forward_quantize": 0}            # few rows need none
    big = cg.Int8MatmulPlan(400, 8, 16)
    assert big.workspace_bytes["forward"] == 0 and g(big._plan, A, 1, A, A, None, A, None, None) == 1
    assert g(p._plan, A + 2, 1, A, A, None, A, A, None) == 3
    quant = L.conv_quantize_rows
    assert quant(None, 1, 4, 4, A, A, None) == 1 and quant(A, 1, 0, 4, A, A, None) == 1
    assert quant(A, 3, 4, 4, A, A, None) == 1 and quant(A, 1, 4, 4, A, A + 4, None) == 3
    assert quant(A, 1, 1 << 30, 1 << 20, A, A, None) == 2


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device behaviour")
def test_without_a_device_calls_fail_loudly():
    L, A = cg.lib(), 256
    n, p = cg.GroupNormPlan(1, 32, 4, 4, 4), cg.Int8MatmulPlan(4, 8, 16)
    assert L.conv_group_norm_forward(n._plan, A, None, None, A, None, A, None) == 4
    assert L.conv_group_norm_forward_int8(n._plan, A, None, None, A, A, None, A, None) == 4
    assert L.conv_group_norm_backward(n._plan, A, A, A, None, None, A, A, A, A, None) == 4
    assert L.conv_int8_forward(p._plan, A, A, A, A, None, A, A, None) == 4
    assert L.conv_int8_forward_quantize(p._plan, A, 1, A, A, None, A, A, None) == 4
    assert L.conv_quantize_rows(A, 1, 4, 4, A, A, None) == 4
    code = ctypes.c_int(5)
    assert L.conv_int8_plan_device_status(p._plan, None, ctypes.byref(code)) == 4 and code.value == 0


def test_binding_refuses_unknown_words():
    with pytest.raises(ValueError):
        cg.GroupNormPlan(1, 32, 4, 4, 4, dtype="f16")
    with pytest.raises(ValueError):
        cg.GroupNormPlan(1, 32, 4, 4, 4, act="gelu")
    with pytest.raises(ValueError):
        cg.Int8MatmulPlan(4, 8, 16, out="int8")
    with pytest.raises(cg.ConvError):
        cg.GroupNormPlan(1, 32, 4, 4, 5)
    with pytest.raises(ValueError):
        cg.group_norm(torch.zeros(1, 2, 2, 32), 4)          # not on the GPU
    with pytest.raises(ValueError):
        cg.int8_matmul(torch.zeros(2, 8, dtype=torch.int8), torch.ones(2), torch.zeros(4, 8, dtype=torch.int8), torch.ones(4))
    with pytest.raises(ValueError):
        cg.quantize_rows(torch.zeros(2, 8))


@pytest.mark.parametrize("args,status", [
    ((1, 1 << 30, 1, 1, 0), 0), ((32, 1 << 30, 1, 1, 0), 0),     # kernels of few rows: any 31-bit number of channels
    ((33, 1 << 30, 1, 1, 0), 2), ((400, 1 << 30, 1, 1, 0), 2),   # tiles: below 2^30
    ((1 << 30, 8, 8, 1, 0), 2), (((1 << 30) - 1, 8, 8, 1, 0), 0),
])
def test_int8_create_at_2_30(args, status):
    L = cg.lib()
    h = ctypes.c_void_p(1234)
    assert L.conv_int8_plan_create(ctypes.byref(h), *args) == status
    if h.value:
        assert L.conv_int8_plan_destroy(h) == 0
