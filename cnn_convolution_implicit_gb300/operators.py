"""Group norm and 8-bit products: ctypes binding of conv_group_norm_*, conv_int8_* and
conv_quantize_rows (include/conv.h).

Argument checks and marshalling only, as in binding.py: every step runs in the library's
CUDA kernels, on torch's current stream or, with ``stream``, as if that were it: results and
workspaces are allocated on it, so torch's allocator reuses them in its order.
"""
from __future__ import annotations

import ctypes

from . import binding
from .binding import CONV_BF16, CONV_F32, ConvError, _plan_status, lib

ACTS = {"none": 0, "relu": 1, "silu": 2}
INT8_KERNELS = {0: "few_rows", 1: "mid_rows", 2: "tiles"}
_DTYPES = {"f32": CONV_F32, "bf16": CONV_BF16}

# torch, imported with the first plan or call (as in binding.py, importing the package needs no
# torch), and what every call takes from it.
_t = None
_raw_stream = None
_current_device = None


def _torch():
    global _t, _raw_stream, _current_device
    if _t is None:
        import torch
        _raw_stream = torch._C._cuda_getCurrentRawStream
        _current_device = torch._C._cuda_getDevice
        _t = torch
    return _t


def _torch_dtypes():
    return {"f32": _torch().float32, "bf16": _torch().bfloat16}


def _choice(value, table, name):
    if value not in table:
        raise ValueError("%s must be one of %s, not %r" % (name, ", ".join(sorted(table)), value))
    return table[value]


def _refuse_device(dev):
    """Raises unless ``dev``, a tensor's device, is the current one: a plan is made for the current
    device, and the library launches there (and refuses a plan of another)."""
    if dev < 0:
        raise ValueError("x must be a CUDA tensor")
    if dev != _current_device():
        raise binding.other_device(dev, _current_device())


def _need(t, name, shape, dtype, dev):
    """A contiguous tensor of that shape and type on CUDA device ``dev``."""
    if t is None or t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on cuda:%d" % (name, dtype, tuple(shape), dev))


def _need_any(t, name, dtypes):
    if not t.is_cuda or t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor of %s" % (name, " or ".join(str(d) for d in dtypes)))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace(nbytes, dev):
    return _t.empty(nbytes, dtype=_t.uint8, device=dev) if nbytes else None


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
        self._L = L
        torch = _torch()
        self.shape, self.C, self.groups = torch.Size((N, H, W, C)), C, groups
        self.dtype, self.torch_dtype, self.eps, self.act = dtype, _torch_dtypes()[dtype], eps, act
        self.stats_shape, self._channels, self._pixels = torch.Size((2, N, groups)), torch.Size((C,)), torch.Size((N * H * W,))
        b = [ctypes.c_ulonglong() for _ in range(3)]
        _check(L.conv_group_norm_workspace(h, *[ctypes.byref(v) for v in b]), "conv_group_norm_workspace")
        self.workspace_bytes = dict(zip(("forward", "forward_int8", "backward"), [v.value for v in b]))

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
        """Checks them; returns x's device."""
        dev = x.get_device()
        if dev < 0 or dev != _current_device():
            _refuse_device(dev)
        _need(x, "x", self.shape, self.torch_dtype, dev)
        if gamma is not None:
            _need(gamma, "gamma", self._channels, _t.float32, dev)
        if beta is not None:
            _need(beta, "beta", self._channels, _t.float32, dev)
        if stats is not None:
            _need(stats, "stats", self.stats_shape, _t.float32, dev)
        return dev

    def forward(self, x, gamma=None, beta=None, y=None, stats=None, stream=None):
        """act(norm(x)); ``stats`` (empty_stats()) receives what backward() reads."""
        if stream is not None:
            with _t.cuda.stream(stream):
                return self.forward(x, gamma, beta, y, stats)
        dev = self._inputs(x, gamma, beta, stats)
        if y is None:
            y = _t.empty_like(x)
        else:
            _need(y, "y", self.shape, self.torch_dtype, dev)
        ws = _workspace(self.workspace_bytes["forward"], dev)
        _check(self._L.conv_group_norm_forward(self._plan, x.data_ptr(), _ptr(gamma), _ptr(beta), y.data_ptr(),
                                               _ptr(stats), _ptr(ws), _raw_stream(dev)), "conv_group_norm_forward")
        return y

    __call__ = forward

    def forward_int8(self, x, gamma=None, beta=None, q=None, scale=None, stats=None, stream=None):
        """(q, scale): act(norm(x)) as int8 [N][H][W][C] with one FP32 scale per pixel [N*H*W]."""
        if stream is not None:
            with _t.cuda.stream(stream):
                return self.forward_int8(x, gamma, beta, q, scale, stats)
        dev = self._inputs(x, gamma, beta, stats)
        if q is None:
            q = _t.empty(self.shape, dtype=_t.int8, device=dev)
        else:
            _need(q, "q", self.shape, _t.int8, dev)
        if scale is None:
            scale = _t.empty(self._pixels, dtype=_t.float32, device=dev)
        else:
            _need(scale, "scale", self._pixels, _t.float32, dev)
        ws = _workspace(self.workspace_bytes["forward_int8"], dev)
        _check(self._L.conv_group_norm_forward_int8(self._plan, x.data_ptr(), _ptr(gamma), _ptr(beta), q.data_ptr(),
                                                    scale.data_ptr(), _ptr(stats), _ptr(ws), _raw_stream(dev)),
               "conv_group_norm_forward_int8")
        return q, scale

    def backward(self, dy, x, stats, gamma=None, beta=None, dx=None, dgamma=None, dbeta=None, stream=None,
                 affine_grads=True):
        """(dx, dgamma, dbeta) from the forward pass's x and stats; without ``affine_grads`` dx alone,
        (dx, None, None)."""
        if stream is not None:
            with _t.cuda.stream(stream):
                return self.backward(dy, x, stats, gamma, beta, dx, dgamma, dbeta, affine_grads=affine_grads)
        if stats is None:
            raise ValueError("stats must be what forward(stats=...) wrote")
        dev = self._inputs(x, gamma, beta, stats)
        _need(dy, "dy", self.shape, self.torch_dtype, dev)
        if dx is None:
            dx = _t.empty_like(x)
        else:
            _need(dx, "dx", self.shape, self.torch_dtype, dev)
        if not affine_grads:
            if dgamma is not None or dbeta is not None:
                raise ValueError("dgamma and dbeta are not written without affine_grads")
        else:
            if dgamma is None:
                dgamma = _t.empty(self._channels, dtype=_t.float32, device=dev)
            else:
                _need(dgamma, "dgamma", self._channels, _t.float32, dev)
            if dbeta is None:
                dbeta = _t.empty(self._channels, dtype=_t.float32, device=dev)
            else:
                _need(dbeta, "dbeta", self._channels, _t.float32, dev)
        ws = _workspace(self.workspace_bytes["backward"], dev)
        _check(self._L.conv_group_norm_backward(self._plan, dy.data_ptr(), x.data_ptr(), stats.data_ptr(), _ptr(gamma),
                                                _ptr(beta), dx.data_ptr(), _ptr(dgamma), _ptr(dbeta),
                                                _ptr(ws), _raw_stream(dev)), "conv_group_norm_backward")
        return dx, dgamma, dbeta

    def empty_stats(self, device="cuda"):
        return _t.empty(self.stats_shape, dtype=_t.float32, device=device)


class Int8MatmulPlan:
    """8-bit product of one shape (include/conv.h, conv_int8_*):
    y[m][n] = act(x_scale[m] * w_scale[n] * sum_k x[m][k] * w[n][k] + bias[n]), x int8 [M][K], w
    int8 [N][K], FP32 scales and bias, y BF16 ("bf16") or FP32 ("f32").  ``x_shape`` [..., K] with M rows
    in all: x has that shape instead, and y [..., N]."""

    def __init__(self, M, N, K, out="bf16", act="none", x_shape=None):
        L = lib()
        self._plan = None
        h = ctypes.c_void_p()
        _check(L.conv_int8_plan_create(ctypes.byref(h), M, N, K, _choice(out, _DTYPES, "out"),
                                       _choice(act, ACTS, "act")), "conv_int8_plan_create")
        self._plan = h
        self._L = L
        torch = _torch()
        self.M, self.N, self.K, self.out, self.act = M, N, K, out, act
        self.torch_dtype = _torch_dtypes()[out]
        self._x = torch.Size((M, K) if x_shape is None else x_shape)
        if self._x.numel() != M * K or self._x[-1] != K:
            raise ValueError("x_shape must hold %d rows of %d" % (M, K))
        self._w, self._y = torch.Size((N, K)), torch.Size(self._x[:-1] + (N,))
        self._rows, self._cols = torch.Size((M,)), torch.Size((N,))
        info = [ctypes.c_int() for _ in range(4)]
        _check(L.conv_int8_plan_info(h, *[ctypes.byref(v) for v in info]), "conv_int8_plan_info")
        self.kernel = INT8_KERNELS[info[0].value]
        self.tile = tuple(v.value for v in info[1:])  # rows, columns, CTAs that share its K ("tiles" alone)
        a, b = ctypes.c_ulonglong(), ctypes.c_ulonglong()
        _check(L.conv_int8_workspace(h, ctypes.byref(a), ctypes.byref(b)), "conv_int8_workspace")
        self.workspace_bytes = {"forward": a.value, "forward_quantize": b.value}

    def close(self):
        if self._plan is not None and binding._lib is not None:
            binding._lib.conv_int8_plan_destroy(self._plan)
        self._plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _operands(self, x, w, w_scale, bias, y):
        """Checks all but x's type; returns x's device."""
        dev = x.get_device()
        if dev < 0 or dev != _current_device():
            _refuse_device(dev)
        _need(x, "x", self._x, x.dtype, dev)
        _need(w, "w", self._w, _t.int8, dev)
        _need(w_scale, "w_scale", self._cols, _t.float32, dev)
        if bias is not None:
            _need(bias, "bias", self._cols, _t.float32, dev)
        if y is not None:
            _need(y, "y", self._y, self.torch_dtype, dev)
        return dev

    def forward(self, x, x_scale, w, w_scale, bias=None, y=None, stream=None):
        """The product of int8 rows x [M][K] with their scales [M]."""
        if stream is not None:
            with _t.cuda.stream(stream):
                return self.forward(x, x_scale, w, w_scale, bias, y)
        if x.dtype is not _t.int8:
            raise ValueError("x must be int8")
        dev = self._operands(x, w, w_scale, bias, y)
        _need(x_scale, "x_scale", self._rows, _t.float32, dev)
        if y is None:
            y = _t.empty(self._y, dtype=self.torch_dtype, device=dev)
        ws = _workspace(self.workspace_bytes["forward"], dev)
        _check(self._L.conv_int8_forward(self._plan, x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
                                         _ptr(bias), y.data_ptr(), _ptr(ws), _raw_stream(dev)), "conv_int8_forward")
        return y

    __call__ = forward

    def forward_quantize(self, x, w, w_scale, bias=None, y=None, stream=None):
        """The product of BF16 or FP32 rows, brought to 8 bits (quantize_rows) in the call."""
        if stream is not None:
            with _t.cuda.stream(stream):
                return self.forward_quantize(x, w, w_scale, bias, y)
        bf16 = x.dtype is _t.bfloat16
        if not bf16 and x.dtype is not _t.float32:
            raise ValueError("x must be bfloat16 or float32")
        dev = self._operands(x, w, w_scale, bias, y)
        if y is None:
            y = _t.empty(self._y, dtype=self.torch_dtype, device=dev)
        ws = _workspace(self.workspace_bytes["forward_quantize"], dev)
        _check(self._L.conv_int8_forward_quantize(self._plan, x.data_ptr(), CONV_BF16 if bf16 else CONV_F32, w.data_ptr(),
                                                  w_scale.data_ptr(), _ptr(bias), y.data_ptr(), _ptr(ws),
                                                  _raw_stream(dev)), "conv_int8_forward_quantize")
        return y

    def device_status(self, stream=None) -> int:
        """Read and clear the plan's own status word, as ConvPlan.device_status."""
        return _plan_status(lib().conv_int8_plan_device_status, self._plan, stream, "conv_int8_plan_device_status")


# ---------------------------------------------------------------- functional forms
_norm_plans = binding.PlanCache()
_int8_plans = binding.PlanCache()


def _norm_plan(x, groups, eps, act):
    key = (x.shape, x.dtype, x.get_device(), groups, eps, act)
    plan = _norm_plans.get(key)
    if plan is None:
        torch = _torch()
        _need_any(x, "x", (torch.bfloat16, torch.float32))
        if x.dim() != 4:
            raise ValueError("x must be an NHWC tensor [N][H][W][C]")
        _refuse_device(x.get_device())
        N, H, W, C = x.shape
        plan = _norm_plans.put(key, GroupNormPlan(N, C, H, W, groups, "bf16" if x.dtype == torch.bfloat16 else "f32",
                                                  eps, act))
    else:
        plan.used = True
    return plan


_norm_fn = None


def _norm_function():
    """The autograd function of group_norm.  It keeps statistics of its own: a caller's buffer may
    hold another call's by the time of the backward pass."""
    global _norm_fn
    if _norm_fn is None:
        from torch.autograd.function import once_differentiable

        class GroupNorm(_torch().autograd.Function):
            @staticmethod
            def forward(ctx, x, gamma, beta, plan):
                stats = plan.empty_stats(x.device)
                y = plan.forward(x, gamma, beta, stats=stats)
                ctx.save_for_backward(x, gamma, beta, stats)
                ctx.mark_non_differentiable(stats)
                ctx.plan = plan
                return y, stats

            @staticmethod
            @once_differentiable
            def backward(ctx, dy, _):
                x, gamma, beta, stats = ctx.saved_tensors
                dy = dy.contiguous()
                if dy.data_ptr() % 16:  # a slice of a larger tensor
                    dy = dy.clone()
                need_x, need_gamma, need_beta, _ = ctx.needs_input_grad
                dx, dgamma, dbeta = ctx.plan.backward(dy, x, stats, gamma, beta, affine_grads=need_gamma or need_beta)
                return dx if need_x else None, dgamma if need_gamma else None, dbeta if need_beta else None, None

        _norm_fn = GroupNorm
    return _norm_fn


def group_norm(x, groups, gamma=None, beta=None, eps=1e-5, act="none", y=None, stats=None, stream=None):
    """act((x - mean) * rstd * gamma + beta) over each image's groups of channels; x NHWC.

    Differentiable: where torch records gradients and x, gamma or beta requires one, the result has
    its backward pass (group_norm_backward; once, and not with ``y`` given).  The plans and the
    8-bit forms record none."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return group_norm(x, groups, gamma, beta, eps, act, y, stats)
    plan = _norm_plan(x, groups, eps, act)
    if (x.requires_grad or (gamma is not None and gamma.requires_grad) or
            (beta is not None and beta.requires_grad)) and _t.is_grad_enabled():
        if y is not None:
            raise ValueError("y cannot be given where the result's gradient is recorded")
        if stats is not None:
            _need(stats, "stats", plan.stats_shape, _t.float32, x.get_device())
        out, own = _norm_function().apply(x, gamma, beta, plan)
        if stats is not None:
            stats.copy_(own)
        return out
    return plan.forward(x, gamma, beta, y, stats)


def group_norm_int8(x, groups, gamma=None, beta=None, eps=1e-5, act="none", stats=None, stream=None):
    """(q, scale): group_norm's result as int8 with one FP32 scale per pixel [N*H*W]."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return group_norm_int8(x, groups, gamma, beta, eps, act, stats)
    return _norm_plan(x, groups, eps, act).forward_int8(x, gamma, beta, stats=stats)


def group_norm_backward(dy, x, stats, groups, gamma=None, beta=None, eps=1e-5, act="none", stream=None):
    """(dx, dgamma, dbeta) of group_norm from its input and the stats it wrote."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return group_norm_backward(dy, x, stats, groups, gamma, beta, eps, act)
    return _norm_plan(x, groups, eps, act).backward(dy, x, stats, gamma, beta)


def _int8_plan(x, w, act, out):
    key = (x.shape, w.shape, x.get_device(), out, act)
    plan = _int8_plans.get(key)
    if plan is None:
        _torch()
        _refuse_device(x.get_device())
        if w.dim() != 2 or x.dim() < 2 or x.shape[-1] != w.shape[1]:
            raise ValueError("x must be [..., K] and w [N][K]: got %s and %s" % (tuple(x.shape), tuple(w.shape)))
        N, K = w.shape
        plan = _int8_plans.put(key, Int8MatmulPlan(x.numel() // K if K else 0, N, K, out, act, x.shape))
    else:
        plan.used = True
    return plan


def int8_matmul(x, x_scale, w, w_scale, bias=None, act="none", out="bf16", stream=None):
    """x int8 [..., K] (rows or NHWC pixels) with x_scale, one FP32 scale per row in row order,
    times w int8 [N][K] with w_scale [N]: [..., N] in ``out`` ("bf16" or "f32")."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return int8_matmul(x, x_scale, w, w_scale, bias, act, out)
    if x_scale.dim() != 1:
        x_scale = x_scale.reshape(-1)
    return _int8_plan(x, w, act, out).forward(x, x_scale, w, w_scale, bias)


def int8_linear(x, w, w_scale, bias=None, act="none", out="bf16", stream=None):
    """x BF16 or FP32 [..., K], its rows brought to 8 bits in the call, times w int8 [N][K]."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return int8_linear(x, w, w_scale, bias, act, out)
    return _int8_plan(x, w, act, out).forward_quantize(x, w, w_scale, bias)


def quantize_rows(x, stream=None):
    """(q, scale): rows of x [..., K] (BF16 or FP32) as int8 with one FP32 scale each, flat."""
    torch = _torch()
    _need_any(x, "x", (torch.bfloat16, torch.float32))
    if x.dim() < 2 or not x.numel():
        raise ValueError("x must be [..., K] with at least one row and one column")
    K = x.shape[-1]
    M = x.numel() // K
    if stream is not None:
        with torch.cuda.stream(stream):
            return quantize_rows(x)
    dev = x.get_device()
    _refuse_device(dev)
    q = torch.empty(x.shape, dtype=torch.int8, device=dev)
    scale = torch.empty(M, dtype=torch.float32, device=dev)
    _check(lib().conv_quantize_rows(x.data_ptr(), CONV_BF16 if x.dtype is torch.bfloat16 else CONV_F32, M, K,
                                    q.data_ptr(), scale.data_ptr(), _raw_stream(dev)), "conv_quantize_rows")
    return q, scale
