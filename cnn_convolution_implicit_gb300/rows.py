"""The residual branch of a layer, on rows (tokens, pixels): the BF16 linear layer, the
root-mean-square norm and dropout; ctypes binding of conv_linear_*, conv_rms_norm_* and conv_dropout
(include/conv.h).

Argument checks and marshalling only, as in operators.py: every step runs in the library's CUDA
kernels, on torch's current stream or, with ``stream``, as if that were it.

A backward pass may be captured into a graph with its forward pass.  As for any operator of torch, no graph recorded
outside of the capture on the same leaves may still be alive then: torch adds to a leaf's gradient on the stream that recorded it
first, and that stream is not the captured one.
"""
from __future__ import annotations

import ctypes

from . import binding, operators as _ops
from .binding import CONV_BF16, CONV_F32, _plan_status, lib
from .operators import ACTS, _DTYPES, _buffer, _check, _choice, _need, _need_any, _ptr, _refuse_device, _refuse_tangents, _torch, _torch_dtypes, _workspace


LINEAR_KERNELS = {0: "few_rows", 1: "tiles"}


def _start():
    """torch, and what every call takes from it.  _t is set last: other threads take the rest to be there with it."""
    global _t, _empty, _empty_like, _bf16, _f32
    if _t is None:
        torch = _torch()
        _empty, _empty_like, _bf16, _f32 = torch.empty, torch.empty_like, torch.bfloat16, torch.float32
        _t = torch
    return _t


_t = _empty = _empty_like = _bf16 = _f32 = None


def _size(n):
    """A size as the library's 32 bits hold it; one past them stays past every limit (ctypes keeps the low bits)."""
    return n if -2 ** 31 <= n < 2 ** 31 else 2 ** 31 - 1


def _upstream(dy):
    """A gradient as autograd hands it over, as the kernels take it."""
    _refuse_tangents(dy)
    dy = dy.contiguous()
    return dy.clone() if dy.data_ptr() % 16 else dy  # a slice of a larger tensor


class _Plan:
    _plan = None

    def close(self):
        if self._plan is not None and binding._lib is not None:
            getattr(binding._lib, self._destroy)(self._plan)
        self._plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class LinearPlan(_Plan):
    """Linear layer of one shape in BF16 (include/conv.h, conv_linear_*):
    z[m][n] = sum_k x[m][k] * w[n][k] + bias[n], y = act(z) + residual, x [M][K], w [N][K], FP32 bias
    [N], residual, y and z [M][N].  ``x_shape`` [..., K] with M rows in all: x has that shape instead, and
    residual, y and z [..., N]."""

    _destroy = "conv_linear_plan_destroy"

    def __init__(self, M, N, K, act="none", x_shape=None):
        L = lib()
        h = ctypes.c_void_p()
        _check(L.conv_linear_plan_create(ctypes.byref(h), _size(M), _size(N), _size(K), _choice(act, ACTS, "act")), "conv_linear_plan_create")
        self._plan = h
        torch = _start()
        self.M, self.N, self.K, self.act = M, N, K, act
        self._x = torch.Size((M, K) if x_shape is None else x_shape)
        if self._x.numel() != M * K or self._x[-1] != K:
            raise ValueError("x_shape must hold %d rows of %d" % (M, K))
        self._w, self._y, self._cols = torch.Size((N, K)), torch.Size(self._x[:-1] + (N,)), torch.Size((N,))
        info = (ctypes.c_int * 8)()
        _check(L.conv_linear_plan_info(h, info), "conv_linear_plan_info")
        self.kernel = LINEAR_KERNELS[info[0]]
        self.tile = tuple(info[1:4])       # rows, columns, units that share its K ("tiles" alone)
        self.grad_tile = tuple(info[4:8])  # of the gradients: rows, columns, dx's and dw's units to a tile
        a, b = ctypes.c_ulonglong(), ctypes.c_ulonglong()
        _check(L.conv_linear_workspace(h, ctypes.byref(a), ctypes.byref(b)), "conv_linear_workspace")
        self.workspace_bytes = {"forward": a.value, "backward": b.value}
        self._forward_bytes, self._backward_bytes = a.value, b.value
        self._forward, self._backward = L.conv_linear_forward, L.conv_linear_backward

    def forward(self, x, w, bias=None, residual=None, y=None, z=None, stream=None):
        """act(x w^T + bias) + residual; ``z`` receives the values before the activation, which backward()
        reads.  ``y`` may be the residual itself, where that is not x too; no other buffer may be shared."""
        if stream is not None:
            with _t.cuda.stream(stream):
                return self.forward(x, w, bias, residual, y, z)
        # The checks stand in line: a call of _need for each tensor took as long as the launch.  (The arguments stay
        # bound to their tensors to the end: a caller's temporaries have no other owner.)
        dev = x.get_device()
        if dev < 0 or dev != _ops._current_device():
            _refuse_device(dev)
        shape = self._y
        if x.shape != self._x or x.dtype is not _bf16 or not x.is_contiguous():
            _need(x, "x", self._x, _bf16, dev)
        if w.shape != self._w or w.dtype is not _bf16 or w.get_device() != dev or not w.is_contiguous():
            _need(w, "w", self._w, _bf16, dev)
        if bias is not None:
            if bias.shape != self._cols or bias.dtype is not _f32 or bias.get_device() != dev or not bias.is_contiguous():
                _need(bias, "bias", self._cols, _f32, dev)
        if residual is not None:
            if residual.shape != shape or residual.dtype is not _bf16 or residual.get_device() != dev or \
                    not residual.is_contiguous():
                _need(residual, "residual", shape, _bf16, dev)
        if z is not None:
            _buffer(z, "z", shape, _bf16, dev)
        if y is None:
            y = _empty(shape, dtype=_bf16, device=dev) if residual is None else _empty_like(residual)
        else:
            _buffer(y, "y", shape, _bf16, dev)
        ws = _workspace(self._forward_bytes, dev) if self._forward_bytes else None
        status = self._forward(self._plan, x.data_ptr(), w.data_ptr(), None if bias is None else bias.data_ptr(),
                               None if residual is None else residual.data_ptr(), y.data_ptr(),
                               None if z is None else z.data_ptr(),
                               None if ws is None else ws.data_ptr(), _ops._raw_stream(dev))
        if status:
            _check(status, "conv_linear_forward")
        return y

    __call__ = forward

    def backward(self, dy, x=None, w=None, z=None, dx=None, dw=None, dbias=None, stream=None, need=(True, True, True)):
        """(dx, dw, dbias) of forward() from its x, w and, with an activation, z; None for those that
        ``need`` (dx, dw, dbias) leaves out.  w is read for dx and x for dw.  The residual's
        gradient is dy itself."""
        if stream is not None:
            with _t.cuda.stream(stream):
                return self.backward(dy, x, w, z, dx, dw, dbias, need=need)
        dev = dy.get_device()
        if dev < 0 or dev != _ops._current_device():
            _refuse_device(dev)
        need_x, need_w, need_b = need
        if dy.shape != self._y or dy.dtype is not _bf16 or not dy.is_contiguous():
            _need(dy, "dy", self._y, _bf16, dev)
        if x is None:
            if need_w:
                _need(x, "x", self._x, _bf16, dev)
        elif x.shape != self._x or x.dtype is not _bf16 or x.get_device() != dev or not x.is_contiguous():
            _need(x, "x", self._x, _bf16, dev)
        if w is None:
            if need_x:
                _need(w, "w", self._w, _bf16, dev)
        elif w.shape != self._w or w.dtype is not _bf16 or w.get_device() != dev or not w.is_contiguous():
            _need(w, "w", self._w, _bf16, dev)
        if z is None:
            if self.act != "none":
                _need(z, "z", self._y, _bf16, dev)
        elif z.shape != self._y or z.dtype is not _bf16 or z.get_device() != dev or not z.is_contiguous():
            _need(z, "z", self._y, _bf16, dev)
        for given, name, shape, dtype, wanted in ((dx, "dx", self._x, _bf16, need_x), (dw, "dw", self._w, _bf16, need_w),
                                                  (dbias, "dbias", self._cols, _f32, need_b)):
            if given is not None:
                if not wanted:
                    raise ValueError("%s is not written without need" % name)
                _buffer(given, name, shape, dtype, dev)
        if dx is None and need_x:
            dx = _empty(self._x, dtype=_bf16, device=dev) if x is None else _empty_like(x)
        if dw is None and need_w:
            dw = _empty(self._w, dtype=_bf16, device=dev) if w is None else _empty_like(w)
        if dbias is None and need_b:
            dbias = _empty(self._cols, dtype=_f32, device=dev)
        ws = _workspace(self._backward_bytes, dev) if self._backward_bytes else None
        status = self._backward(self._plan, dy.data_ptr(), _ptr(x), _ptr(w), _ptr(z), _ptr(dx), _ptr(dw), _ptr(dbias),
                                None if ws is None else ws.data_ptr(), _ops._raw_stream(dev))
        if status:
            _check(status, "conv_linear_backward")
        return dx, dw, dbias

    def device_status(self, stream=None) -> int:
        """Read and clear the plan's own status word, as ConvPlan.device_status."""
        return _plan_status(lib().conv_linear_plan_device_status, self._plan, stream, "conv_linear_plan_device_status")


class RmsNormPlan(_Plan):
    """Root-mean-square norm of M rows of C values (include/conv.h, conv_rms_norm_*) in FP32 ("f32") or
    BF16 ("bf16"): h = x + residual, y = h / sqrt(mean(h^2) + eps) * gamma, FP32 gamma [C] (None: 1).
    ``x_shape`` [..., C] with M rows in all: x, residual, y and h have that shape.  rstd is FP32 [M]."""

    _destroy = "conv_rms_norm_plan_destroy"

    def __init__(self, M, C, dtype="bf16", eps=1e-6, x_shape=None):
        L = lib()
        h = ctypes.c_void_p()
        _check(L.conv_rms_norm_plan_create(ctypes.byref(h), _size(M), _size(C), eps, _choice(dtype, _DTYPES, "dtype")),
               "conv_rms_norm_plan_create")
        self._plan = h
        torch = _start()
        self.M, self.C, self.dtype, self.torch_dtype, self.eps = M, C, dtype, _torch_dtypes()[dtype], eps
        self.shape = torch.Size((M, C) if x_shape is None else x_shape)
        if self.shape.numel() != M * C or self.shape[-1] != C:
            raise ValueError("x_shape must hold %d rows of %d" % (M, C))
        self._cols, self._rows = torch.Size((C,)), torch.Size((M,))
        b = ctypes.c_ulonglong()
        _check(L.conv_rms_norm_workspace(h, ctypes.byref(b)), "conv_rms_norm_workspace")
        self.workspace_bytes = {"backward": b.value}

        self._forward, self._forward_int8 = L.conv_rms_norm_forward, L.conv_rms_norm_forward_int8
        self._backward, self._backward_bytes = L.conv_rms_norm_backward, b.value

    def _inputs(self, x, gamma, residual, h, rstd):
        """Checks them; returns x's device and h, made where a residual calls for one."""
        dev, shape, dtype = x.get_device(), self.shape, self.torch_dtype
        if dev < 0 or dev != _ops._current_device():
            _refuse_device(dev)
        if x.shape != shape or x.dtype is not dtype or not x.is_contiguous():
            _need(x, "x", shape, dtype, dev)
        if gamma is not None and (gamma.shape != self._cols or gamma.dtype is not _f32 or gamma.get_device() != dev or
                                  not gamma.is_contiguous()):
            _need(gamma, "gamma", self._cols, _f32, dev)
        if residual is not None:
            if residual.shape != shape or residual.dtype is not dtype or residual.get_device() != dev or \
                    not residual.is_contiguous():
                _need(residual, "residual", shape, dtype, dev)
            if h is None:
                h = _empty_like(x)
            else:
                _buffer(h, "h", shape, dtype, dev)
        elif h is not None:
            raise ValueError("h is written with a residual alone: without one it is x")
        if rstd is not None:
            _buffer(rstd, "rstd", self._rows, _f32, dev)
        return dev, h

    def forward(self, x, gamma=None, residual=None, y=None, h=None, rstd=None, stream=None):
        """y, or (y, h) with a residual; ``rstd`` (empty_rstd()) receives what backward() reads.  ``h`` may be
        the residual itself."""
        if stream is not None:
            with _t.cuda.stream(stream):
                return self.forward(x, gamma, residual, y, h, rstd)
        dev, h = self._inputs(x, gamma, residual, h, rstd)
        if y is None:
            y = _empty_like(x)
        else:
            _buffer(y, "y", self.shape, self.torch_dtype, dev)
        status = self._forward(self._plan, x.data_ptr(), None if residual is None else residual.data_ptr(),
                               None if gamma is None else gamma.data_ptr(), y.data_ptr(), None if h is None else h.data_ptr(),
                               None if rstd is None else rstd.data_ptr(), _ops._raw_stream(dev))
        if status:
            _check(status, "conv_rms_norm_forward")
        return y if residual is None else (y, h)

    __call__ = forward

    def forward_int8(self, x, gamma=None, residual=None, q=None, scale=None, h=None, rstd=None, stream=None):
        """(q, scale), or (q, scale, h) with a residual: y as int8 with one FP32 scale per row [M]."""
        if stream is not None:
            with _t.cuda.stream(stream):
                return self.forward_int8(x, gamma, residual, q, scale, h, rstd)
        dev, h = self._inputs(x, gamma, residual, h, rstd)
        if q is None:
            q = _empty(self.shape, dtype=_t.int8, device=dev)
        else:
            _buffer(q, "q", self.shape, _t.int8, dev)
        if scale is None:
            scale = _empty(self._rows, dtype=_f32, device=dev)
        else:
            _buffer(scale, "scale", self._rows, _f32, dev)
        status = self._forward_int8(self._plan, x.data_ptr(), _ptr(residual), _ptr(gamma), q.data_ptr(), scale.data_ptr(),
                                    _ptr(h), _ptr(rstd), _ops._raw_stream(dev))
        if status:
            _check(status, "conv_rms_norm_forward_int8")
        return (q, scale) if residual is None else (q, scale, h)

    def backward(self, dy, h, rstd, gamma=None, dh=None, dx=None, dgamma=None, stream=None, gamma_grad=True):
        """(dx, dgamma) from forward()'s h (x without a residual) and rstd; ``dh`` is the gradient of its
        output h, dx that of x and of the residual alike.  Without ``gamma_grad`` (dx, None).  ``dx`` may be dy
        or dh itself."""
        if stream is not None:
            with _t.cuda.stream(stream):
                return self.backward(dy, h, rstd, gamma, dh, dx, dgamma, gamma_grad=gamma_grad)
        dev, shape, dtype = dy.get_device(), self.shape, self.torch_dtype
        if dev < 0 or dev != _ops._current_device():
            _refuse_device(dev)
        if dy.shape != shape or dy.dtype is not dtype or not dy.is_contiguous():
            _need(dy, "dy", shape, dtype, dev)
        if h.shape != shape or h.dtype is not dtype or h.get_device() != dev or not h.is_contiguous():
            _need(h, "h", shape, dtype, dev)
        _need(rstd, "rstd", self._rows, _f32, dev)
        if gamma is not None:
            _need(gamma, "gamma", self._cols, _f32, dev)
        if dh is not None:
            _need(dh, "dh", shape, dtype, dev)
        if dx is None:
            dx = _empty_like(dy)
        else:
            _buffer(dx, "dx", shape, dtype, dev)
        ws = None
        if gamma_grad:
            if dgamma is None:
                dgamma = _empty(self._cols, dtype=_f32, device=dev)
            else:
                _buffer(dgamma, "dgamma", self._cols, _f32, dev)
            ws = _workspace(self._backward_bytes, dev) if self._backward_bytes else None
        elif dgamma is not None:
            raise ValueError("dgamma is not written without gamma_grad")
        status = self._backward(self._plan, dy.data_ptr(), h.data_ptr(), rstd.data_ptr(), _ptr(gamma), _ptr(dh), dx.data_ptr(),
                                _ptr(dgamma), _ptr(ws), _ops._raw_stream(dev))
        if status:
            _check(status, "conv_rms_norm_backward")
        return dx, dgamma

    def empty_rstd(self, device="cuda"):
        return _empty(self._rows, dtype=_f32, device=device)


# ---------------------------------------------------------------- functional forms
_linear_plans = binding.PlanCache()
_rms_plans = binding.PlanCache()
_functions = {}
_TWO = (2,)


def _linear_plan(x, w, act):
    key = (x.shape, w.shape, x.get_device(), act)
    plan = _linear_plans.get(key)
    if plan is None:
        _start()
        _refuse_device(x.get_device())
        if w.dim() != 2 or x.dim() < 2 or x.shape[-1] != w.shape[1]:
            raise ValueError("x must be [..., K] and w [N][K]: got %s and %s" % (tuple(x.shape), tuple(w.shape)))
        N, K = w.shape
        plan = _linear_plans.put(key, LinearPlan(x.numel() // K if K else 0, N, K, act, x.shape))
    else:
        plan.used = True
    return plan


def _rms_plan(x, eps):
    key = (x.shape, x.dtype, x.get_device(), eps)
    plan = _rms_plans.get(key)
    if plan is None:
        torch = _start()
        _need_any(x, "x", (torch.bfloat16, torch.float32))
        if x.dim() < 2:
            raise ValueError("x must be [..., C]")
        _refuse_device(x.get_device())
        C = x.shape[-1]
        plan = _rms_plans.put(key, RmsNormPlan(x.numel() // C if C else 0, C, "bf16" if x.dtype is torch.bfloat16 else "f32",
                                               eps, x.shape))
    else:
        plan.used = True
    return plan


def _function(name):
    """The autograd functions of linear, rms_norm and dropout.  They keep buffers of their own: a caller's
    may hold another call's by the time of the backward pass."""
    if not _functions:
        torch = _start()
        from torch.autograd.function import once_differentiable

        class Linear(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, w, bias, residual, plan):
                need_x, need_w, need_b = ctx.needs_input_grad[:3]
                z = torch.empty(plan._y, dtype=x.dtype, device=x.device) if plan.act != "none" and (need_x or need_w or need_b) else None
                y = plan.forward(x, w, bias, residual, z=z)
                ctx.save_for_backward(x if need_w else None, w if need_x else None, z)  # what the gradients wanted read
                ctx.plan = plan
                return y

            @staticmethod
            @once_differentiable
            def backward(ctx, dy):
                x, w, z = ctx.saved_tensors
                need = ctx.needs_input_grad
                dx = dw = dbias = None
                if any(need[:3]):
                    dx, dw, dbias = ctx.plan.backward(_upstream(dy), x, w, z, need=need[:3])
                return dx, dw, dbias, dy if need[3] else None, None

        class RmsNorm(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, gamma, residual, plan):
                rstd = plan.empty_rstd(x.device)
                out = plan.forward(x, gamma, residual, rstd=rstd)
                ctx.save_for_backward(x if residual is None else out[1], gamma, rstd)
                ctx.mark_non_differentiable(rstd)
                ctx.set_materialize_grads(False)  # an output that nobody used would bring a gradient of zeros to write and read
                ctx.plan = plan
                return (out, rstd) if residual is None else out + (rstd,)

            @staticmethod
            @once_differentiable
            def backward(ctx, dy, *more):
                h, gamma, rstd = ctx.saved_tensors
                need_x, need_gamma, need_r, _ = ctx.needs_input_grad
                dh = _upstream(more[0]) if len(more) > 1 and more[0] is not None else None
                if dy is not None:
                    dx, dgamma = ctx.plan.backward(_upstream(dy), h, rstd, gamma, dh, gamma_grad=need_gamma)
                else:  # y played no part
                    dx, dgamma = dh, torch.zeros_like(gamma) if need_gamma else None
                return dx if need_x else None, dgamma, dx if need_r else None, None

        class Dropout(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, residual, p, state):
                state = state.clone()  # the caller's may have moved on by the time of the backward pass
                ctx.save_for_backward(state)
                ctx.p = p
                return _dropout(x, p, state, residual)

            @staticmethod
            @once_differentiable
            def backward(ctx, dy):
                state, = ctx.saved_tensors
                need = ctx.needs_input_grad
                return _dropout(_upstream(dy), ctx.p, state) if need[0] else None, dy if need[1] else None, None, None

        _functions.update(linear=Linear, rms_norm=RmsNorm, dropout=Dropout)
    return _functions[name]


def linear(x, w, bias=None, act="none", residual=None, y=None, z=None, stream=None):
    """act(x w^T + bias) + residual in BF16: x [..., K], w [N][K], FP32 bias [N], residual [..., N]; act
    "none", "relu" or "silu".  ``z`` receives the values before the activation, which linear_backward reads; ``y``,
    the result's buffer, may be the residual itself, where that is not x too.

    Differentiable: where torch records gradients and x, w, bias or residual requires one, the result
    has its backward pass (once, and not with ``y`` or ``z`` given).  The plans record none.  A tensor with a
    forward-mode tangent is refused."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return linear(x, w, bias, act, residual, y, z)
    plan = _linear_plan(x, w, act)
    _refuse_tangents(x, w, bias, residual)
    if (x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad) or
            (residual is not None and residual.requires_grad)) and _t.is_grad_enabled():
        if y is not None or z is not None:
            raise ValueError("y and z cannot be given where the result's gradient is recorded")
        return _function("linear").apply(x, w, bias, residual, plan)
    return plan.forward(x, w, bias, residual, y, z)


def linear_backward(dy, x, w, z=None, act="none", stream=None):
    """(dx, dw, dbias) of linear from its x and w and, with an activation, the z it wrote; the
    residual's gradient is dy itself."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return linear_backward(dy, x, w, z, act)
    plan = _linear_plan(x, w, act)
    _refuse_tangents(dy, x, w, z)
    return plan.backward(dy, x, w, z)


def rms_norm(x, gamma=None, residual=None, eps=1e-6, h=None, rstd=None, stream=None):
    """y = h / sqrt(mean(h^2) + eps) * gamma over the last axis of h = x + residual, in x's type; x
    [..., C] BF16 or FP32, FP32 gamma [C].  Returns y, or (y, h) with a residual.  ``h``, that result's buffer, may be
    the residual itself; ``rstd`` FP32 [rows] receives what rms_norm_backward reads.

    Differentiable: where torch records gradients and x, gamma or residual requires one, the results
    have their backward pass (once, and not with ``h`` given).  The plans and the 8-bit form
    record none.  A tensor with a forward-mode tangent is refused."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return rms_norm(x, gamma, residual, eps, h, rstd)
    plan = _rms_plan(x, eps)
    _refuse_tangents(x, gamma, residual)
    if (x.requires_grad or (gamma is not None and gamma.requires_grad) or
            (residual is not None and residual.requires_grad)) and _t.is_grad_enabled():
        if h is not None:
            raise ValueError("h cannot be given where the result's gradient is recorded")
        if rstd is not None:
            _need(rstd, "rstd", plan._rows, _f32, x.get_device())
        *out, own = _function("rms_norm").apply(x, gamma, residual, plan)
        if rstd is not None:
            rstd.copy_(own)
        return out[0] if residual is None else tuple(out)
    return plan.forward(x, gamma, residual, h=h, rstd=rstd)


def rms_norm_int8(x, gamma=None, residual=None, eps=1e-6, h=None, rstd=None, stream=None):
    """(q, scale), or (q, scale, h) with a residual: rms_norm's result as int8 with one FP32 scale per
    row [rows], as int8_matmul takes it."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return rms_norm_int8(x, gamma, residual, eps, h, rstd)
    return _rms_plan(x, eps).forward_int8(x, gamma, residual, h=h, rstd=rstd)


def rms_norm_backward(dy, h, rstd, gamma=None, dh=None, stream=None):
    """(dx, dgamma) of rms_norm from the h (x without a residual) and rstd it wrote; ``dh`` is the gradient of
    its output h.  dx is the gradient of x and of the residual alike."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return rms_norm_backward(dy, h, rstd, gamma, dh)
    plan = _rms_plan(h, 1e-6)  # eps is in rstd already
    _refuse_tangents(dy, h, rstd, gamma, dh)
    return plan.backward(dy, h, rstd, gamma, dh)


def _dropout(x, p, state, residual=None, y=None):
    dtype, shape, dev = x.dtype, x.shape, x.get_device()
    if (dtype is not _bf16 and dtype is not _f32) or dev < 0 or not x.is_contiguous():
        _need_any(x, "x", (_bf16, _f32))
    if dev != _ops._current_device():
        _refuse_device(dev)
    if residual is not None:
        if residual.shape != shape or residual.dtype is not dtype or residual.get_device() != dev or \
                not residual.is_contiguous():
            _need(residual, "residual", shape, dtype, dev)
    if state.dtype is not _t.int64 or state.shape != _TWO or state.get_device() != dev or not state.is_contiguous():
        _need(state, "state", _TWO, _t.int64, dev)
    if y is None:
        y = _empty_like(x)
    else:
        _buffer(y, "y", shape, dtype, dev)
    status = (binding._lib or lib()).conv_dropout(x.data_ptr(), None if residual is None else residual.data_ptr(),
                                                  CONV_BF16 if dtype is _bf16 else CONV_F32, x.numel(), p, state.data_ptr(),
                                                  y.data_ptr(), _ops._raw_stream(dev))
    if status:
        _check(status, "conv_dropout")
    return y


def dropout(x, p, state, residual=None, y=None, stream=None):
    """x / (1 - p) where the generator keeps an element, 0 where it drops one (with probability p), plus
    the residual; x BF16 or FP32 of any shape.  ``state`` is an int64 tensor of two on the GPU, seed and offset, read when
    the kernel runs: the same state gives the same mask, and a program moves the offset (or the seed)
    on for a new one, in a captured graph too.  (Where a forward pass is run a second time for its backward pass, as
    checkpointing does, it has to find the state of the first.)  ``y``, the result's buffer, may be x or the residual itself.

    Differentiable: where torch records gradients and x or residual requires one, the result has its
    backward pass (dropout_backward; once, and not with ``y`` given).  A tensor with a forward-mode
    tangent is refused."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return dropout(x, p, state, residual, y)
    if _t is None:
        _start()
    _refuse_tangents(x, residual)
    if (x.requires_grad or (residual is not None and residual.requires_grad)) and _t.is_grad_enabled():
        if y is not None:
            raise ValueError("y cannot be given where the result's gradient is recorded")
        if state.dtype is not _t.int64 or state.shape != _TWO:
            raise ValueError("state must be an int64 tensor of two")
        return _function("dropout").apply(x, residual, p, state)
    return _dropout(x, p, state, residual, y)


def dropout_backward(dy, p, state, stream=None):
    """The gradient of dropout's x: the same mask and factor on dy (the residual's gradient is dy itself)."""
    return dropout(dy, p, state, stream=stream)
