"""Group norm and 8-bit products: ctypes binding of conv_group_norm_*, conv_int8_* and
conv_quantize_rows (include/conv.h).

Argument checks and marshalling only, as in binding.py: every step runs in the library's
CUDA kernels, on the given stream or torch's current one.  Results and workspaces are
allocated on that stream, so torch's allocator reuses them in its order.
"""
from __future__ import annotations

import contextlib
import ctypes

from . import binding
from .binding import CONV_BF16, CONV_F32, ConvError, _plan_status, lib

ACTS = {"none": 0, "relu": 1, "silu": 2}
_DTYPES = {"f32": CONV_F32, "bf16": CONV_BF16}


def _torch_dtypes():
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}


def _choice(value, table, name):
    if value not in table:
        raise ValueError("%s must be one of %s, not %r" % (name, ", ".join(sorted(table)), value))
    return table[value]


def _need(t, name, shape, dtype, device):
    if t is None or t.dtype != dtype or t.device != device or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s" % (name, dtype, tuple(shape), device))


def _need_any(t, name, dtypes):
    if not t.is_cuda or t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor of %s" % (name, " or ".join(str(d) for d in dtypes)))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(stream):
    """(the stream to launch on, a context that allocates on it)."""
    import torch
    if stream is None:
        return None, contextlib.nullcontext()
    return stream, torch.cuda.stream(stream)


def _handle(stream, device):
    import torch
    return (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream


def _check(status, what):
    if status != 0:
        raise ConvError(status, what)


class GroupNormPlan:
    """Group norm with an activation over NHWC maps of one shape (include/conv.h,
    conv_group_norm_*): x [N][H][W][C] in FP32 ("f32") or BF16 ("bf16"), FP32 gamma and beta
    [C] (None: 1 and 0), act "none", "relu" or "silu".  stats is FP32 [2][N][groups]: means,
    then reciprocal standard deviations."""

    def __init__(self, N, C, H, W, groups, dtype="bf16", eps=1e-5, act="none"):
        L = lib()
        self._plan = None
        h = ctypes.c_void_p()
        _check(L.conv_group_norm_plan_create(ctypes.byref(h), N, C, H, W, groups, eps,
                                             _choice(dtype, _DTYPES, "dtype"), _choice(act, ACTS, "act")),
               "conv_group_norm_plan_create")
        self._plan = h
        self.shape, self.C, self.groups = (N, H, W, C), C, groups
        self.dtype, self.torch_dtype, self.eps, self.act = dtype, _torch_dtypes()[dtype], eps, act
        self.stats_shape = (2, N, groups)
        b = ctypes.c_ulonglong()
        _check(L.conv_group_norm_workspace(h, ctypes.byref(b)), "conv_group_norm_workspace")
        self.workspace_bytes = b.value

    def close(self):
        if self._plan is not None and binding._lib is not None:
            binding._lib.conv_group_norm_plan_destroy(self._plan)
        self._plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _inputs(self, x, gamma, beta, stats):
        import torch
        if not x.is_cuda:
            raise ValueError("x must be a CUDA tensor")
        _need(x, "x", self.shape, self.torch_dtype, x.device)
        for t, name in ((gamma, "gamma"), (beta, "beta")):
            if t is not None:
                _need(t, name, (self.C,), torch.float32, x.device)
        if stats is not None:
            _need(stats, "stats", self.stats_shape, torch.float32, x.device)

    def _workspace(self, device):
        import torch
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)

    def forward(self, x, gamma=None, beta=None, y=None, stats=None, stream=None):
        """act(norm(x)); ``stats`` (empty_stats()) receives what backward() reads."""
        import torch
        self._inputs(x, gamma, beta, stats)
        stream, scope = _on(stream)
        with scope:
            if y is None:
                y = torch.empty_like(x)
            else:
                _need(y, "y", self.shape, self.torch_dtype, x.device)
            ws = self._workspace(x.device)
            _check(lib().conv_group_norm_forward(self._plan, x.data_ptr(), _ptr(gamma), _ptr(beta), y.data_ptr(),
                                                 _ptr(stats), ws.data_ptr(), _handle(stream, x.device)),
                   "conv_group_norm_forward")
        return y

    __call__ = forward

    def forward_int8(self, x, gamma=None, beta=None, q=None, scale=None, stats=None, stream=None):
        """(q, scale): act(norm(x)) as int8 [N][H][W][C] with one FP32 scale per pixel [N*H*W]."""
        import torch
        self._inputs(x, gamma, beta, stats)
        N, H, W, _ = self.shape
        stream, scope = _on(stream)
        with scope:
            if q is None:
                q = torch.empty(self.shape, dtype=torch.int8, device=x.device)
            else:
                _need(q, "q", self.shape, torch.int8, x.device)
            if scale is None:
                scale = torch.empty(N * H * W, dtype=torch.float32, device=x.device)
            else:
                _need(scale, "scale", (N * H * W,), torch.float32, x.device)
            ws = self._workspace(x.device)
            _check(lib().conv_group_norm_forward_int8(self._plan, x.data_ptr(), _ptr(gamma), _ptr(beta), q.data_ptr(),
                                                      scale.data_ptr(), _ptr(stats), ws.data_ptr(),
                                                      _handle(stream, x.device)),
                   "conv_group_norm_forward_int8")
        return q, scale

    def backward(self, dy, x, stats, gamma=None, beta=None, dx=None, dgamma=None, dbeta=None, stream=None):
        """(dx, dgamma, dbeta) from the forward pass's x and stats."""
        import torch
        if stats is None:
            raise ValueError("stats must be what forward(stats=...) wrote")
        self._inputs(x, gamma, beta, stats)
        _need(dy, "dy", self.shape, self.torch_dtype, x.device)
        stream, scope = _on(stream)
        with scope:
            if dx is None:
                dx = torch.empty_like(x)
            else:
                _need(dx, "dx", self.shape, self.torch_dtype, x.device)
            grads = []
            for t, name in ((dgamma, "dgamma"), (dbeta, "dbeta")):
                if t is None:
                    t = torch.empty(self.C, dtype=torch.float32, device=x.device)
                else:
                    _need(t, name, (self.C,), torch.float32, x.device)
                grads.append(t)
            ws = self._workspace(x.device)
            _check(lib().conv_group_norm_backward(self._plan, dy.data_ptr(), x.data_ptr(), stats.data_ptr(),
                                                  _ptr(gamma), _ptr(beta), dx.data_ptr(), grads[0].data_ptr(),
                                                  grads[1].data_ptr(), ws.data_ptr(), _handle(stream, x.device)),
                   "conv_group_norm_backward")
        return dx, grads[0], grads[1]

    def empty_stats(self, device="cuda"):
        import torch
        return torch.empty(self.stats_shape, dtype=torch.float32, device=device)


class Int8MatmulPlan:
    """8-bit product of one shape (include/conv.h, conv_int8_*):
    y[m][n] = act(x_scale[m] * w_scale[n] * sum_k x[m][k] * w[n][k] + bias[n]), x int8 [M][K], w
    int8 [N][K], FP32 scales and bias, y BF16 ("bf16") or FP32 ("f32")."""

    def __init__(self, M, N, K, out="bf16", act="none"):
        L = lib()
        self._plan = None
        h = ctypes.c_void_p()
        _check(L.conv_int8_plan_create(ctypes.byref(h), M, N, K, _choice(out, _DTYPES, "out"),
                                       _choice(act, ACTS, "act")), "conv_int8_plan_create")
        self._plan = h
        self.M, self.N, self.K, self.out, self.act = M, N, K, out, act
        self.torch_dtype = _torch_dtypes()[out]
        b = ctypes.c_ulonglong()
        _check(L.conv_int8_workspace(h, ctypes.byref(b)), "conv_int8_workspace")
        self.workspace_bytes = b.value

    def close(self):
        if self._plan is not None and binding._lib is not None:
            binding._lib.conv_int8_plan_destroy(self._plan)
        self._plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _weights(self, w, w_scale, bias, device):
        import torch
        _need(w, "w", (self.N, self.K), torch.int8, device)
        _need(w_scale, "w_scale", (self.N,), torch.float32, device)
        if bias is not None:
            _need(bias, "bias", (self.N,), torch.float32, device)

    def _output(self, y, device):
        import torch
        if y is None:
            return torch.empty((self.M, self.N), dtype=self.torch_dtype, device=device)
        _need(y, "y", (self.M, self.N), self.torch_dtype, device)
        return y

    def forward(self, x, x_scale, w, w_scale, bias=None, y=None, stream=None):
        """The product of int8 rows x [M][K] with their scales [M]."""
        import torch
        _need_any(x, "x", (torch.int8,))
        _need(x, "x", (self.M, self.K), torch.int8, x.device)
        _need(x_scale, "x_scale", (self.M,), torch.float32, x.device)
        self._weights(w, w_scale, bias, x.device)
        stream, scope = _on(stream)
        with scope:
            y = self._output(y, x.device)
            _check(lib().conv_int8_forward(self._plan, x.data_ptr(), x_scale.data_ptr(), w.data_ptr(),
                                           w_scale.data_ptr(), _ptr(bias), y.data_ptr(), _handle(stream, x.device)),
                   "conv_int8_forward")
        return y

    __call__ = forward

    def forward_quantize(self, x, w, w_scale, bias=None, y=None, stream=None):
        """The product of BF16 or FP32 rows, brought to 8 bits (quantize_rows) in the call."""
        import torch
        _need_any(x, "x", (torch.bfloat16, torch.float32))
        _need(x, "x", (self.M, self.K), x.dtype, x.device)
        self._weights(w, w_scale, bias, x.device)
        stream, scope = _on(stream)
        with scope:
            y = self._output(y, x.device)
            ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=x.device) if self.workspace_bytes else None
            _check(lib().conv_int8_forward_quantize(self._plan, x.data_ptr(),
                                                    CONV_BF16 if x.dtype == torch.bfloat16 else CONV_F32,
                                                    w.data_ptr(), w_scale.data_ptr(), _ptr(bias), y.data_ptr(),
                                                    _ptr(ws), _handle(stream, x.device)),
                   "conv_int8_forward_quantize")
        return y

    def device_status(self, stream=None) -> int:
        """Read and clear the plan's own status word, as ConvPlan.device_status."""
        return _plan_status(lib().conv_int8_plan_device_status, self._plan, stream, "conv_int8_plan_device_status")


# ---------------------------------------------------------------- functional forms
_norm_plans = {}
_int8_plans = {}


def _norm_plan(x, groups, eps, act):
    import torch
    _need_any(x, "x", (torch.bfloat16, torch.float32))
    if x.dim() != 4:
        raise ValueError("x must be an NHWC tensor [N][H][W][C]")
    key = (x.device.index, x.shape, x.dtype, groups, eps, act)
    plan = _norm_plans.get(key)
    if plan is None:
        N, H, W, C = x.shape
        plan = _norm_plans[key] = GroupNormPlan(N, C, H, W, groups, "bf16" if x.dtype == torch.bfloat16 else "f32",
                                                eps, act)
    return plan


def group_norm(x, groups, gamma=None, beta=None, eps=1e-5, act="none", y=None, stats=None, stream=None):
    """act((x - mean) * rstd * gamma + beta) over each image's groups of channels; x NHWC."""
    return _norm_plan(x, groups, eps, act).forward(x, gamma, beta, y, stats, stream)


def group_norm_int8(x, groups, gamma=None, beta=None, eps=1e-5, act="none", stats=None, stream=None):
    """(q, scale): group_norm's result as int8 with one FP32 scale per pixel [N*H*W]."""
    return _norm_plan(x, groups, eps, act).forward_int8(x, gamma, beta, stats=stats, stream=stream)


def group_norm_backward(dy, x, stats, groups, gamma=None, beta=None, eps=1e-5, act="none", stream=None):
    """(dx, dgamma, dbeta) of group_norm from its input and the stats it wrote."""
    return _norm_plan(x, groups, eps, act).backward(dy, x, stats, gamma, beta, stream=stream)


def _int8_plan(x, w, act, out):
    if w.dim() != 2 or x.dim() < 2 or x.shape[-1] != w.shape[1]:
        raise ValueError("x must be [..., K] and w [N][K]: got %s and %s" % (tuple(x.shape), tuple(w.shape)))
    N, K = w.shape
    M = x.numel() // K if K else 0
    key = (x.device.index, M, N, K, out, act)
    plan = _int8_plans.get(key)
    if plan is None:
        plan = _int8_plans[key] = Int8MatmulPlan(M, N, K, out, act)
    return plan


def _as_rows(x, plan):
    return x if x.dim() == 2 else x.view(plan.M, plan.K)


def _as_given(y, x):
    return y if x.dim() == 2 else y.view(*x.shape[:-1], y.shape[1])


def int8_matmul(x, x_scale, w, w_scale, bias=None, act="none", out="bf16", stream=None):
    """x int8 [..., K] (rows or NHWC pixels) with x_scale, one FP32 scale per row in row order,
    times w int8 [N][K] with w_scale [N]: [..., N] in ``out`` ("bf16" or "f32")."""
    import torch
    _need_any(x, "x", (torch.int8,))
    plan = _int8_plan(x, w, act, out)
    return _as_given(plan.forward(_as_rows(x, plan), x_scale.view(-1), w, w_scale, bias, stream=stream), x)


def int8_linear(x, w, w_scale, bias=None, act="none", out="bf16", stream=None):
    """x BF16 or FP32 [..., K], its rows brought to 8 bits in the call, times w int8 [N][K]."""
    import torch
    _need_any(x, "x", (torch.bfloat16, torch.float32))
    plan = _int8_plan(x, w, act, out)
    return _as_given(plan.forward_quantize(_as_rows(x, plan), w, w_scale, bias, stream=stream), x)


def quantize_rows(x, stream=None):
    """(q, scale): rows of x [..., K] (BF16 or FP32) as int8 with one FP32 scale each, flat."""
    import torch
    _need_any(x, "x", (torch.bfloat16, torch.float32))
    if x.dim() < 2 or not x.numel():
        raise ValueError("x must be [..., K] with at least one row and one column")
    K = x.shape[-1]
    M = x.numel() // K
    stream, scope = _on(stream)
    with scope:
        q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
        scale = torch.empty(M, dtype=torch.float32, device=x.device)
        _check(lib().conv_quantize_rows(x.data_ptr(), CONV_BF16 if x.dtype == torch.bfloat16 else CONV_F32, M, K,
                                        q.data_ptr(), scale.data_ptr(), _handle(stream, x.device)),
               "conv_quantize_rows")
    return q, scale
