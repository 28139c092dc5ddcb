"""The dense tower's operators (``include/tbe_tower.h``): layer norm, linear layers on rows grouped
by expert, AdamW over many tensors.

Argument marshalling as in the package's other functions: torch tensors in, the C entry point of
the same name called on the current stream, TbeError where it refuses.  What the C interface cannot
see, a tensor's shape, strides, type and device, is checked here.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Union

import torch

from . import _I_DTYPE, _W_DTYPE, TbeError, _check, lib

TBE_LAYER_NORM_MAX_WIDTH = 1 << 24
TBE_STATE_F32, TBE_STATE_8BIT = 0, 1
TBE_ADAMW_BLOCK = 128   # values of an 8-bit state that share a scale
TBE_ADAMW_CONTROL = 4   # doubles of a control tensor: step, lr factor, gradient factor, skip


class tbe_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("exp_avg_scale", ctypes.c_void_p), ("exp_avg_sq_scale", ctypes.c_void_p),
                ("numel", ctypes.c_int64), ("weight_decay", ctypes.c_float),
                ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("state", ctypes.c_int32)]


# The checks build their messages only when they refuse: a call of a small kernel takes a few
# microseconds in all.
def _device() -> int:
    return torch.cuda.current_device() if torch.cuda.is_initialized() or torch.cuda.is_available() else -2


def _current(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _refuse(what: str):
    raise TbeError(what)


def _off_gpu(name: str, t: torch.Tensor):
    _refuse(f"{name} is on {t.device}, not on the current GPU")


def _dtype(name: str, t: torch.Tensor) -> int:
    d = _W_DTYPE.get(t.dtype)
    if d is None:
        _refuse(f"{name} is {t.dtype}: float32, float16 or bfloat16 are supported")
    return d


def _rows(name: str, t: torch.Tensor, dev: int, shape=None) -> int:
    """The row stride of a matrix whose rows are contiguous."""
    if t.get_device() != dev:
        _off_gpu(name, t)
    s = t.shape
    if len(s) != 2 or (shape is not None and s != shape):
        _refuse(f"{name} has shape {tuple(s)}" + ("" if shape is None else f", not {tuple(shape)}"))
    ld, one = t.stride()
    if one != 1 and s[1] > 1 and s[0] > 0:
        _refuse(f"{name}: rows have to be contiguous")
    return ld if s[0] > 1 else s[1]


def _whole(name: str, t: torch.Tensor, dev: int, shape, dtype=None):
    """A contiguous tensor of this shape (and type)."""
    if t.get_device() != dev:
        _off_gpu(name, t)
    if t.shape != shape or not t.is_contiguous():
        _refuse(f"{name} has shape {tuple(t.shape)} and strides {tuple(t.stride())}: contiguous {tuple(shape)} is needed")
    if dtype is not None and t.dtype != dtype:
        _refuse(f"{name} is {t.dtype}, not {dtype}")


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _bytes(workspace: Optional[torch.Tensor], dev: int) -> int:
    if workspace is None:
        return 0
    if workspace.get_device() != dev:
        _off_gpu("workspace", workspace)
    return workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def _vectors(dev: int, width: int, *named) -> int:
    """The one type of the vectors that are given."""
    wd, dtype, shape = 0, None, (width,)
    for name, t in named:
        if t is not None:
            _whole(name, t, dev, shape, dtype)
            if dtype is None:
                dtype, wd = t.dtype, _dtype(name, t)
    return wd


def tbe_layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor],
                           eps: float, y: torch.Tensor, mean: Optional[torch.Tensor] = None,
                           rstd: Optional[torch.Tensor] = None, stream=None):
    """y = (x - mean) * rstd * weight + bias for each row of x [rows, width]."""
    dev = _device()
    xs = _rows("x", x, dev)
    rows, width = shape = x.shape
    ys = _rows("y", y, dev, shape)
    wd = _vectors(dev, width, ("weight", weight), ("bias", bias))
    if mean is not None:
        _whole("mean", mean, dev, (rows,), torch.float32)
    if rstd is not None:
        _whole("rstd", rstd, dev, (rows,), torch.float32)
    st = lib().tbe_layer_norm_forward(rows, width, x.data_ptr(), xs, _dtype("x", x), _at(weight), _at(bias), wd, eps,
                                      y.data_ptr(), ys, _dtype("y", y), _at(mean), _at(rstd), _current(stream, dev))
    _check(st, "tbe_layer_norm_forward")


def tbe_layer_norm_backward_workspace_bytes(rows: int, width: int) -> int:
    return int(lib().tbe_layer_norm_backward_workspace_bytes(int(rows), int(width)))


def tbe_layer_norm_backward(x: torch.Tensor, grad_y: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                            weight: Optional[torch.Tensor], grad_x: Optional[torch.Tensor],
                            grad_weight: Optional[torch.Tensor], grad_bias: Optional[torch.Tensor],
                            workspace: Optional[torch.Tensor], stream=None):
    """The gradients of tbe_layer_norm_forward; each of the three may be left out (None)."""
    dev = _device()
    xs = _rows("x", x, dev)
    rows, width = shape = x.shape
    gs = _rows("grad_y", grad_y, dev, shape)
    os = 0
    if grad_x is not None:
        os = _rows("grad_x", grad_x, dev, shape)
        if grad_x.dtype != x.dtype:
            _refuse(f"grad_x is {grad_x.dtype}, not {x.dtype}")
    wd = _vectors(dev, width, ("weight", weight), ("grad_weight", grad_weight), ("grad_bias", grad_bias))
    _whole("mean", mean, dev, (rows,), torch.float32)
    _whole("rstd", rstd, dev, (rows,), torch.float32)
    st = lib().tbe_layer_norm_backward(rows, width, x.data_ptr(), xs, _dtype("x", x), grad_y.data_ptr(), gs,
                                       _dtype("grad_y", grad_y), mean.data_ptr(), rstd.data_ptr(), _at(weight), wd,
                                       _at(grad_x), os, _at(grad_weight), _at(grad_bias), _at(workspace),
                                       _bytes(workspace, dev), _current(stream, dev))
    _check(st, "tbe_layer_norm_backward")


# ---------------------------------------------------------------------------
# linear layers on rows grouped by expert
# ---------------------------------------------------------------------------
def _grouped(shape, offsets: torch.Tensor, dev: int):
    if len(shape) != 3:
        _refuse(f"weights have shape {tuple(shape)}, not (experts, outer, inner)")
    ot = _I_DTYPE.get(offsets.dtype)
    if ot is None:
        _refuse(f"offsets are {offsets.dtype}: int32 or int64 are supported")
    _whole("offsets", offsets, dev, (shape[0] + 1,))
    return ot


def _same(name: str, t: torch.Tensor, first: str, dtype):
    if t.dtype != dtype:
        _refuse(f"{name} is not of {first}'s type")


def tbe_grouped_linear_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                               offsets: torch.Tensor, y: torch.Tensor, stream=None):
    """y[i] = weight[e] @ x[i] + bias[e] for offsets[e] <= i < offsets[e + 1]; zero behind the last."""
    dev = _device()
    ot = _grouped(weight.shape, offsets, dev)
    experts, outer, inner = weight.shape
    rows = x.shape[0]
    xs, ys = _rows("x", x, dev, (rows, inner)), _rows("y", y, dev, (rows, outer))
    _whole("weight", weight, dev, weight.shape)
    _same("weight", weight, "x", x.dtype)
    if bias is not None:
        _whole("bias", bias, dev, (experts, outer))
        _same("bias", bias, "x", x.dtype)
    st = lib().tbe_grouped_linear_forward(rows, experts, inner, outer, x.data_ptr(), xs, weight.data_ptr(), _at(bias),
                                          _dtype("x", x), offsets.data_ptr(), ot, y.data_ptr(), ys, _dtype("y", y),
                                          _current(stream, dev))
    _check(st, "tbe_grouped_linear_forward")


def tbe_grouped_linear_backward_input(grad_y: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor,
                                      grad_x: torch.Tensor, stream=None):
    """grad_x[i] = grad_y[i] @ weight[e]."""
    dev = _device()
    ot = _grouped(weight.shape, offsets, dev)
    experts, outer, inner = weight.shape
    rows = grad_y.shape[0]
    gs, xs = _rows("grad_y", grad_y, dev, (rows, outer)), _rows("grad_x", grad_x, dev, (rows, inner))
    _whole("weight", weight, dev, weight.shape)
    _same("weight", weight, "grad_y", grad_y.dtype)
    st = lib().tbe_grouped_linear_backward_input(rows, experts, inner, outer, grad_y.data_ptr(), gs, weight.data_ptr(),
                                                 _dtype("grad_y", grad_y), offsets.data_ptr(), ot, grad_x.data_ptr(), xs,
                                                 _dtype("grad_x", grad_x), _current(stream, dev))
    _check(st, "tbe_grouped_linear_backward_input")


def tbe_grouped_linear_backward_weight_workspace_bytes(rows: int, experts: int, inner: int, outer: int) -> int:
    return int(lib().tbe_grouped_linear_backward_weight_workspace_bytes(int(rows), int(experts), int(inner),
                                                                        int(outer)))


def tbe_grouped_linear_backward_weight(x: torch.Tensor, grad_y: torch.Tensor, offsets: torch.Tensor,
                                       grad_weight: torch.Tensor, grad_bias: Optional[torch.Tensor],
                                       workspace: Optional[torch.Tensor], stream=None):
    """grad_weight[e] = the sum of outer products of expert e's rows, grad_bias[e] their grad_y's sum."""
    dev = _device()
    ot = _grouped(grad_weight.shape, offsets, dev)
    experts, outer, inner = grad_weight.shape
    rows = x.shape[0]
    xs, gs = _rows("x", x, dev, (rows, inner)), _rows("grad_y", grad_y, dev, (rows, outer))
    _whole("grad_weight", grad_weight, dev, grad_weight.shape)
    _same("grad_y", grad_y, "x", x.dtype)
    if grad_bias is not None:
        _whole("grad_bias", grad_bias, dev, (experts, outer), grad_weight.dtype)
    st = lib().tbe_grouped_linear_backward_weight(rows, experts, inner, outer, x.data_ptr(), xs, grad_y.data_ptr(), gs,
                                                  _dtype("x", x), offsets.data_ptr(), ot, grad_weight.data_ptr(),
                                                  _at(grad_bias), _dtype("grad_weight", grad_weight), _at(workspace),
                                                  _bytes(workspace, dev), _current(stream, dev))
    _check(st, "tbe_grouped_linear_backward_weight")


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
class AdamWTensors:
    """The tensors of a step, as an array of tbe_adamw_tensor on the host (the tensors are kept alive
    here).  States are float32, or uint8 codes with uint8 scales of ceil(numel / TBE_ADAMW_BLOCK)
    bytes.  A step reads the gradients from the buffers given here; a program whose gradients are new
    tensors at every step hands them over with set_gradients before it."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                 exp_avg: Sequence[torch.Tensor], exp_avg_sq: Sequence[torch.Tensor],
                 weight_decay: Union[float, Sequence[float]] = 0.0,
                 masters: Optional[Sequence[Optional[torch.Tensor]]] = None,
                 exp_avg_scales: Optional[Sequence[Optional[torch.Tensor]]] = None,
                 exp_avg_sq_scales: Optional[Sequence[Optional[torch.Tensor]]] = None):
        n, dev = len(params), _device()
        self.device = dev
        none = [None] * n
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else list(weight_decay)
        self.tensors = [list(x) if x is not None else none for x in
                        (params, grads, exp_avg, exp_avg_sq, masters, exp_avg_scales, exp_avg_sq_scales)]
        if any(len(x) != n for x in self.tensors) or len(decay) != n:
            _refuse(f"{n} params need as many gradients, states and weight decays")
        self.c = (tbe_adamw_tensor * max(1, n))()
        self.count = n
        self.numels = [p.numel() for p in params]
        for i, (p, g, m, v, w, ms, vs) in enumerate(zip(*self.tensors)):
            numel = p.numel()
            eight = m.dtype == torch.uint8
            st = torch.uint8 if eight else torch.float32
            blocks = -(-numel // TBE_ADAMW_BLOCK)
            for name, t, size, dt in (("param", p, numel, None), ("gradient", g, numel, None),
                                      ("exp_avg", m, numel, st), ("exp_avg_sq", v, numel, st),
                                      ("master", w, numel, torch.float32), ("exp_avg_scale", ms, blocks, torch.uint8),
                                      ("exp_avg_sq_scale", vs, blocks, torch.uint8)):
                if t is None:
                    if eight and "scale" in name:
                        _refuse(f"tensor {i}: states of 8 bits need scales")
                    continue
                if t.get_device() != dev or not t.is_contiguous() or t.numel() != size or (dt is not None and t.dtype != dt):
                    self._refuse_tensor(i, name, t, size, dt)
            self.c[i] = tbe_adamw_tensor(
                p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), None if w is None else w.data_ptr(),
                ms.data_ptr() if eight else None, vs.data_ptr() if eight else None, numel, decay[i],
                _dtype(f"tensor {i}: param", p), _dtype(f"tensor {i}: gradient", g),
                TBE_STATE_8BIT if eight else TBE_STATE_F32)

    def _refuse_tensor(self, i, name, t, size, dtype):
        if t.get_device() != self.device:
            _off_gpu(f"tensor {i}: {name}", t)
        _refuse(f"tensor {i}: {name} is {t.dtype} of {t.numel()} with strides {tuple(t.stride())}: "
                f"contiguous {'' if dtype is None else dtype} of {size} is needed")

    def set_gradients(self, grads: Sequence[torch.Tensor]):
        """Takes these gradients in place of the ones before, all or none of them."""
        grads = list(grads)
        if len(grads) != self.count:
            _refuse(f"{self.count} params need as many gradients")
        types = []
        for i, (g, numel) in enumerate(zip(grads, self.numels)):
            if g.get_device() != self.device or not g.is_contiguous() or g.numel() != numel:
                self._refuse_tensor(i, "gradient", g, numel, None)
            types.append(_dtype(f"tensor {i}: gradient", g))
        for c, g, dtype in zip(self.c, grads, types):
            c.grad, c.grad_dtype = g.data_ptr(), dtype
        self.tensors[1] = grads


def _same_device(tensors: AdamWTensors, dev: int):
    if tensors.device != dev:
        _refuse(f"the tensors are on GPU {tensors.device}, the current one is {dev}")


def tbe_adamw_step(tensors: AdamWTensors, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                   eps: float = 1e-8, control: Optional[torch.Tensor] = None, stream=None):
    """One AdamW step on every tensor.  control (float64, on the GPU): step, lr factor, gradient
    factor, skip; its step takes the place of `step`."""
    dev = _device()
    _same_device(tensors, dev)
    if control is not None:
        _whole("control", control, dev, (TBE_ADAMW_CONTROL,), torch.float64)
    st = lib().tbe_adamw_step(tensors.c, tensors.count, step, lr, beta1, beta2, eps, _at(control), _current(stream, dev))
    _check(st, "tbe_adamw_step")


def tbe_adamw_state_read(tensors: AdamWTensors, exp_avg_out: Sequence[torch.Tensor],
                         exp_avg_sq_out: Sequence[torch.Tensor], stream=None):
    """The values of states of 8 bits, into float32 tensors or bfloat16 ones (exact from 2^-126 on)."""
    n, dev, c = tensors.count, _device(), tensors.c
    _same_device(tensors, dev)
    if len(exp_avg_out) != n or len(exp_avg_sq_out) != n:
        _refuse(f"{n} tensors need as many outputs of each state")
    dtype = exp_avg_out[0].dtype if n else torch.float32
    array = ctypes.c_void_p * max(1, n)
    arrays = []
    T = torch.Tensor
    for outs in (exp_avg_out, exp_avg_sq_out):
        if list(map(T.numel, outs)) != tensors.numels or set(map(T.get_device, outs)) - {dev} \
                or set(map(T.dtype.__get__, outs)) - {dtype} or not all(map(T.is_contiguous, outs)):
            for i, t in enumerate(outs):
                if t.get_device() != dev:
                    _off_gpu(f"output {i}", t)
                if t.numel() != c[i].numel or t.dtype != dtype or not t.is_contiguous():
                    _refuse(f"output {i} is {t.dtype} of {t.numel()}: contiguous {dtype} of {c[i].numel} is needed")
        arrays.append(array(*map(T.data_ptr, outs)))
    st = lib().tbe_adamw_state_read(c, n, *arrays, _dtype("output 0", exp_avg_out[0]) if n else 0, _current(stream, dev))
    _check(st, "tbe_adamw_state_read")
