"""Host-side checks of the linear layer, the root-mean-square norm and dropout (no GPU needed): shapes,
flags and pointers are refused with their status before anything is launched, tensors of another
device before anything is planned; the oracle's generator gives its published vectors."""
import ctypes

import numpy as np
import pytest
import torch

import cnn_convolution_implicit_gb300 as cg
import row_refs as ref
from cnn_convolution_implicit_gb300 import operators, rows
from test_devices import OnDevice

NAN, INF = float("nan"), float("inf")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("args,status", [
    ((0, 8, 1e-6, 1), 1), ((8, 0, 1e-6, 1), 1), ((8, -3, 1e-6, 1), 1), ((8, 8, -1e-6, 1), 1), ((8, 8, NAN, 1), 1),
    ((8, 8, INF, 1), 1), ((8, 8, 1e-6, 2), 1), ((1, (1 << 20) + 1, 1e-6, 1), 2), ((1 << 30, 8, 1e-6, 1), 2),
    (((1 << 30) - 1, 2048, 1e-6, 1), 2), ((1, 1, 0.0, 0), 0), ((1, 1 << 20, 1e-6, 1), 0), (((1 << 30) - 1, 1, 1e-6, 0), 0),
])
def test_rms_norm_create(args, status):
    L = cg.lib()
    h = ctypes.c_void_p(1234)
    assert L.conv_rms_norm_plan_create(ctypes.byref(h), *args) == status
    assert (h.value is None) == (status != 0)
    if h.value:
        assert L.conv_rms_norm_plan_destroy(h) == 0


@pytest.mark.parametrize("args,status", [
    ((0, 8, 8, 0), 1), ((8, 0, 8, 0), 1), ((8, 8, -1, 0), 1), ((8, 8, 8, 3), 1), ((1 << 29, 8, 8, 0), 2), ((8, 1 << 29, 8, 0), 2),
    ((8, 8, 1 << 29, 0), 2), (((1 << 29) - 1, 8, 4096, 0), 2), (((1 << 29) - 1, 4096, 8, 0), 2), ((1, 1, 1, 2), 0),
    ((1, 1 << 20, 1 << 20, 1), 0), (((1 << 29) - 1, 1, 1, 0), 0), ((1, (1 << 29) - 1, 1, 0), 0), ((1, 1, (1 << 29) - 1, 0), 0),
])
def test_linear_create(args, status):
    L = cg.lib()
    h = ctypes.c_void_p(1234)
    assert L.conv_linear_plan_create(ctypes.byref(h), *args) == status
    assert (h.value is None) == (status != 0)
    if h.value:
        assert L.conv_linear_plan_destroy(h) == 0


def test_null_and_misaligned_pointers():
    L, A = cg.lib(), 256
    assert L.conv_rms_norm_plan_create(None, 8, 8, 1e-6, 1) == 1 and L.conv_linear_plan_create(None, 8, 8, 8, 0) == 1
    assert L.conv_rms_norm_plan_destroy(None) == 0 and L.conv_linear_plan_destroy(None) == 0
    assert L.conv_rms_norm_workspace(None, None) == 1 and L.conv_linear_workspace(None, None, None) == 1
    assert L.conv_linear_plan_device_status(None, None, None) == 1
    n = cg.RmsNormPlan(4, 32)
    fwd, q8, bwd = L.conv_rms_norm_forward, L.conv_rms_norm_forward_int8, L.conv_rms_norm_backward
    assert fwd(None, A, None, None, A, None, None, None) == 1
    assert fwd(n._plan, None, None, None, A, None, None, None) == 1
    assert fwd(n._plan, A, None, None, None, None, None, None) == 1
    assert fwd(n._plan, A, None, None, A, A, None, None) == 1                     # h without a residual
    for bad in ((A + 2, A, A, A, A, A), (A, A + 8, A, A, A, A), (A, A, A + 4, A, A, A), (A, A, A, A + 8, A, A),
                (A, A, A, A, A + 2, A), (A, A, A, A, A, A + 4)):
        assert fwd(n._plan, *bad, None) == 3
    assert q8(n._plan, A, None, None, A, None, None, None, None) == 1
    assert q8(n._plan, A, None, None, None, A, None, None, None) == 1
    assert q8(n._plan, A, None, None, A + 8, A, None, None, None) == 3
    assert bwd(n._plan, A, A, None, None, None, A, None, A, None) == 1            # no rstd
    many = cg.RmsNormPlan(4000, 32)
    assert n.workspace_bytes["backward"] == 0 and many.workspace_bytes["backward"] > 0
    assert bwd(many._plan, A, A, A, None, None, A, A, None, None) == 1            # dgamma without a workspace
    assert bwd(n._plan, A, A, A, None, None, A + 2, A, A, None) == 3
    p, a = cg.LinearPlan(400, 16, 32, "none"), cg.LinearPlan(400, 16, 32, "silu")
    assert L.conv_linear_plan_info(None, A) == 1 and L.conv_linear_plan_info(p._plan, None) == 1
    f, b = L.conv_linear_forward, L.conv_linear_backward
    ws = A if p.workspace_bytes["forward"] else None
    assert f(None, A, A, None, None, A, None, A, None) == 1
    for null in ((None, A, None, None, A, None), (A, None, None, None, A, None), (A, A, None, None, None, None)):
        assert f(p._plan, *null, ws, None) == 1
    for bad in ((A + 2, A, A, A, A, A), (A, A + 8, A, A, A, A), (A, A, A + 4, A, A, A), (A, A, A, A + 2, A, A),
                (A, A, A, A, A + 2, A), (A, A, A, A, A, A + 2)):
        assert f(p._plan, *bad, A, None) == 3
    odd = cg.LinearPlan(400, 17, 33, "none")
    if odd.workspace_bytes["forward"]:
        assert f(odd._plan, A, A, None, None, A, None, None, None) == 1
    assert b(p._plan, None, A, A, None, A, A, A, A, None) == 1
    assert b(p._plan, A, A, A, None, None, None, None, A, None) == 1              # nothing wanted
    assert b(p._plan, A, A, None, None, A, A, A, A, None) == 1                    # dx without w
    assert b(p._plan, A, None, A, None, A, A, A, A, None) == 1                    # dw without x
    assert b(a._plan, A, A, A, None, A, A, A, A, None) == 1                       # an activation without z
    assert a.workspace_bytes["backward"] > 0 and b(a._plan, A, A, A, A, A, A, A, None, None) == 1
    assert b(a._plan, A, A, A, A + 2, A, A, A, A, None) == 3
    d = L.conv_dropout
    assert d(None, None, 1, 8, 0.1, A, A, None) == 1 and d(A, None, 1, 8, 0.1, None, A, None) == 1
    assert d(A, None, 1, 8, 0.1, A, None, None) == 1 and d(A, None, 1, 0, 0.1, A, A, None) == 1
    for p_bad in (-0.01, 1.01, NAN, INF):
        assert d(A, None, 1, 8, p_bad, A, A, None) == 1
    assert d(A, None, 2, 8, 0.1, A, A, None) == 1 and d(A, None, 1, (1 << 40) + 1, 0.1, A, A, None) == 2
    assert d(A + 2, None, 1, 8, 0.1, A, A, None) == 3 and d(A, A + 8, 1, 8, 0.1, A, A, None) == 3
    assert d(A, None, 1, 8, 0.1, A + 4, A, None) == 3 and d(A, None, 1, 8, 0.1, A, A + 2, None) == 3


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device behaviour")
def test_without_a_device_calls_fail_loudly():
    L, A = cg.lib(), 256
    n, p = cg.RmsNormPlan(4, 32), cg.LinearPlan(4, 8, 16)
    assert L.conv_rms_norm_forward(n._plan, A, None, None, A, None, None, None) == 4
    assert L.conv_rms_norm_forward_int8(n._plan, A, None, None, A, A, None, None, None) == 4
    assert L.conv_rms_norm_backward(n._plan, A, A, A, None, None, A, A, A, None) == 4
    assert L.conv_linear_forward(p._plan, A, A, None, None, A, None, A, None) == 4
    assert L.conv_linear_backward(p._plan, A, A, A, None, A, A, A, A, None) == 4
    assert L.conv_dropout(A, None, 1, 8, 0.1, A, A, None) == 4
    code = ctypes.c_int(5)
    assert L.conv_linear_plan_device_status(p._plan, None, ctypes.byref(code)) == 4 and code.value == 0


def test_binding_refuses():
    for make in (lambda: cg.LinearPlan(4, 8, 16, act="gelu"), lambda: cg.RmsNormPlan(4, 8, dtype="f16"),
                 lambda: cg.LinearPlan(4, 8, 16, x_shape=(2, 3, 16)), lambda: cg.RmsNormPlan(4, 8, x_shape=(2, 3, 8)),
                 lambda: cg.linear(torch.zeros(2, 8, dtype=BF16), torch.zeros(4, 8, dtype=BF16)),      # not on the GPU
                 lambda: cg.rms_norm(torch.zeros(2, 8)), lambda: cg.rms_norm_int8(torch.zeros(2, 8)),
                 lambda: cg.dropout(torch.zeros(2, 8), 0.1, torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            make()
    for make in (lambda: cg.LinearPlan(0, 8, 16), lambda: cg.RmsNormPlan(4, 0), lambda: cg.RmsNormPlan(4, 8, eps=-1.0)):
        with pytest.raises(cg.ConvError):
            make()


@pytest.mark.parametrize("past", [1 << 31, (1 << 32) + 5, (1 << 33) + 8])
def test_sizes_past_32_bits_are_refused(past):
    """Not taken for what their low bits hold."""
    for make in (lambda: cg.LinearPlan(past, 8, 8), lambda: cg.LinearPlan(8, past, 8), lambda: cg.LinearPlan(8, 8, past),
                 lambda: cg.RmsNormPlan(past, 8), lambda: cg.RmsNormPlan(8, past)):
        with pytest.raises(cg.ConvError):
            make()


def _calls(i):
    x, w, y = OnDevice((4, 16), BF16, i), OnDevice((8, 16), BF16, i), OnDevice((4, 8), BF16, i)
    rstd, state = OnDevice((4,), F32, i), OnDevice((2,), torch.int64, i)
    for t in (x, w, y, rstd, state):
        t.requires_grad = False
    return {
        "linear": lambda: cg.linear(x, w), "linear_backward": lambda: cg.linear_backward(y, x, w),
        "rms_norm": lambda: cg.rms_norm(x), "rms_norm_int8": lambda: cg.rms_norm_int8(x),
        "rms_norm_backward": lambda: cg.rms_norm_backward(x, x, rstd),
        "dropout": lambda: cg.dropout(x, 0.1, state), "dropout_backward": lambda: cg.dropout_backward(x, 0.1, state),
        "LinearPlan.forward": lambda: cg.LinearPlan(4, 8, 16).forward(x, w),
        "LinearPlan.backward": lambda: cg.LinearPlan(4, 8, 16).backward(y, x, w),
        "RmsNormPlan.forward": lambda: cg.RmsNormPlan(4, 16).forward(x),
        "RmsNormPlan.forward_int8": lambda: cg.RmsNormPlan(4, 16).forward_int8(x),
        "RmsNormPlan.backward": lambda: cg.RmsNormPlan(4, 16).backward(x, x, rstd),
    }


@pytest.mark.parametrize("name", sorted(_calls(1)))
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    operators._torch()
    monkeypatch.setattr(operators, "_current_device", lambda: 0)
    rows._linear_plans.clear()
    rows._rms_plans.clear()
    with pytest.raises(ValueError, match="cuda:0 is current"):
        _calls(1)[name]()
    assert not rows._linear_plans and not rows._rms_plans


@pytest.mark.parametrize("counter,key,want", [
    # the known answers published with the generator (ten rounds)
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_the_oracles_generator(counter, key, want):
    assert [int(v) for v in ref.philox([np.array(c) for c in counter], key)] == list(want)


def _variants():
    """The kernels and tiles that the GPU tests' sizes run (the plans choose alike without a device)."""
    from test_gpu_linear import GRAD_SIZES, SIZES
    forward, grads = set(), set()
    for M, N, K in SIZES:
        p = cg.LinearPlan(M, N, K)
        forward.add((p.kernel, p.tile[1], p.tile[2], N % 8 == 0, K % 8 == 0))
    for M, N, K in GRAD_SIZES:
        rows_, cols, dx, dw = cg.LinearPlan(M, N, K).grad_tile
        grads.add((cols, dx > 1, dw > 1, K % 8 == 0))
    return forward, grads


@pytest.mark.skipif(torch.cuda.is_available(), reason="counted for 152 SMs")
def test_the_gpu_tests_reach_every_kernel():
    forward, grads = _variants()
    for aligned in (True, False):
        assert any(f[0] == "few_rows" and f[4] == aligned for f in forward)
        for columns in (64, 128, 256):
            for split in (1, 2, 4, 8) if columns < 256 else (1,):      # pairs share a K rarely: once is enough
                assert any(f[0] == "tiles" and f[1:4] == (columns, split, aligned) for f in forward), (columns, split, aligned)
            assert any(g[0] == columns and g[3] == aligned for g in grads), (columns, aligned)
    assert any(f[1] == 256 and f[2] > 1 for f in forward)
    assert any(f[1] == 64 and f[2] == 3 for f in forward)        # parts in the workspace, not a cluster
    assert any(g[1] and not g[2] for g in grads) and any(g[2] and not g[1] for g in grads) and any(g[1] and g[2] for g in grads)
