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

from . import _I_DTYPE, _W_DTYPE, TbeError, _check, _ptr, _stream, lib

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


def _need(ok: bool, what: str):
    if not ok:
        raise TbeError(what)


def _on_gpu(name: str, t: torch.Tensor):
    _need(t.is_cuda and t.device.index == torch.cuda.current_device(),
          f"{name} is on {t.device}, not on the current GPU")


def _dtype(name: str, t: torch.Tensor) -> int:
    _need(t.dtype in _W_DTYPE, f"{name} is {t.dtype}: float32, float16 or bfloat16 are supported")
    return _W_DTYPE[t.dtype]


def _rows(name: str, t: torch.Tensor, shape=None) -> int:
    """The row stride of a matrix whose rows are contiguous."""
    _on_gpu(name, t)
    _need(t.dim() == 2 and (shape is None or tuple(t.shape) == tuple(shape)),
          f"{name} has shape {tuple(t.shape)}" + ("" if shape is None else f", not {tuple(shape)}"))
    _need(t.shape[1] <= 1 or t.shape[0] == 0 or t.stride(1) == 1, f"{name}: rows have to be contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _whole(name: str, t: torch.Tensor, shape, dtype=None):
    """A contiguous tensor of this shape (and type)."""
    _on_gpu(name, t)
    _need(tuple(t.shape) == tuple(shape) and t.is_contiguous(),
          f"{name} has shape {tuple(t.shape)} and strides {tuple(t.stride())}: contiguous {tuple(shape)} is needed")
    _need(dtype is None or t.dtype == dtype, f"{name} is {t.dtype}, not {dtype}")


def _bytes(workspace: Optional[torch.Tensor]) -> int:
    if workspace is None:
        return 0
    _on_gpu("workspace", workspace)
    return workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def tbe_layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor],
                           eps: float, y: torch.Tensor, mean: Optional[torch.Tensor] = None,
                           rstd: Optional[torch.Tensor] = None, stream=None):
    """y = (x - mean) * rstd * weight + bias for each row of x [rows, width]."""
    xs = _rows("x", x)
    rows, width = x.shape
    ys = _rows("y", y, x.shape)
    vectors = [("weight", weight), ("bias", bias)]
    wd = _vectors(vectors, width)
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is not None:
            _whole(name, t, (rows,), torch.float32)
    st = lib().tbe_layer_norm_forward(rows, width, _ptr(x), xs, _dtype("x", x), _ptr(weight), _ptr(bias), wd,
                                      float(eps), _ptr(y), ys, _dtype("y", y), _ptr(mean), _ptr(rstd),
                                      _stream(stream))
    _check(st, "tbe_layer_norm_forward")


def _vectors(named, width: int) -> int:
    """The one type of the vectors that are given."""
    wd, first = 0, None
    for name, t in named:
        if t is None:
            continue
        first = t if first is None else first
        _whole(name, t, (width,), first.dtype)
        wd = _dtype(name, t)
    return wd


def tbe_layer_norm_backward_workspace_bytes(rows: int, width: int) -> int:
    return int(lib().tbe_layer_norm_backward_workspace_bytes(int(rows), int(width)))


def tbe_layer_norm_backward(x: torch.Tensor, grad_y: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                            weight: Optional[torch.Tensor], grad_x: Optional[torch.Tensor],
                            grad_weight: Optional[torch.Tensor], grad_bias: Optional[torch.Tensor],
                            workspace: Optional[torch.Tensor], stream=None):
    xs = _rows("x", x)
    rows, width = x.shape
    gs = _rows("grad_y", grad_y, x.shape)
    os = 0
    if grad_x is not None:
        os = _rows("grad_x", grad_x, x.shape)
        _need(grad_x.dtype == x.dtype, f"grad_x is {grad_x.dtype}, not {x.dtype}")
    wd = _vectors([("weight", weight), ("grad_weight", grad_weight), ("grad_bias", grad_bias)], width)
    _whole("mean", mean, (rows,), torch.float32)
    _whole("rstd", rstd, (rows,), torch.float32)
    st = lib().tbe_layer_norm_backward(rows, width, _ptr(x), xs, _dtype("x", x), _ptr(grad_y), gs,
                                       _dtype("grad_y", grad_y), _ptr(mean), _ptr(rstd), _ptr(weight), wd,
                                       _ptr(grad_x), os, _ptr(grad_weight), _ptr(grad_bias), _ptr(workspace),
                                       _bytes(workspace), _stream(stream))
    _check(st, "tbe_layer_norm_backward")


# ---------------------------------------------------------------------------
# linear layers on rows grouped by expert
# ---------------------------------------------------------------------------
def _grouped(weight_shape, offsets: torch.Tensor):
    _need(len(weight_shape) == 3, f"weights have shape {tuple(weight_shape)}, not (experts, outer, inner)")
    experts, outer, inner = weight_shape
    _need(offsets.dtype in _I_DTYPE, f"offsets are {offsets.dtype}: int32 or int64 are supported")
    _whole("offsets", offsets, (experts + 1,))
    return experts, outer, inner


def _same(named):
    first = named[0]
    for name, t in named[1:]:
        _need(t is None or t.dtype == first[1].dtype, f"{name} is not of {first[0]}'s type")


def tbe_grouped_linear_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                               offsets: torch.Tensor, y: torch.Tensor, stream=None):
    """y[i] = weight[e] @ x[i] + bias[e] for offsets[e] <= i < offsets[e + 1]; zero behind the last."""
    experts, outer, inner = _grouped(weight.shape, offsets)
    rows = x.shape[0]
    xs, ys = _rows("x", x, (rows, inner)), _rows("y", y, (rows, outer))
    _whole("weight", weight, weight.shape)
    if bias is not None:
        _whole("bias", bias, (experts, outer))
    _same([("x", x), ("weight", weight), ("bias", bias)])
    st = lib().tbe_grouped_linear_forward(rows, experts, inner, outer, _ptr(x), xs, _ptr(weight), _ptr(bias),
                                          _dtype("x", x), _ptr(offsets), _I_DTYPE[offsets.dtype], _ptr(y), ys,
                                          _dtype("y", y), _stream(stream))
    _check(st, "tbe_grouped_linear_forward")


def tbe_grouped_linear_backward_input(grad_y: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor,
                                      grad_x: torch.Tensor, stream=None):
    """grad_x[i] = grad_y[i] @ weight[e]."""
    experts, outer, inner = _grouped(weight.shape, offsets)
    rows = grad_y.shape[0]
    gs, xs = _rows("grad_y", grad_y, (rows, outer)), _rows("grad_x", grad_x, (rows, inner))
    _whole("weight", weight, weight.shape)
    _same([("grad_y", grad_y), ("weight", weight)])
    st = lib().tbe_grouped_linear_backward_input(rows, experts, inner, outer, _ptr(grad_y), gs, _ptr(weight),
                                                 _dtype("grad_y", grad_y), _ptr(offsets),
                                                 _I_DTYPE[offsets.dtype], _ptr(grad_x), xs,
                                                 _dtype("grad_x", grad_x), _stream(stream))
    _check(st, "tbe_grouped_linear_backward_input")


def tbe_grouped_linear_backward_weight_workspace_bytes(rows: int, experts: int, inner: int, outer: int) -> int:
    return int(lib().tbe_grouped_linear_backward_weight_workspace_bytes(int(rows), int(experts), int(inner),
                                                                        int(outer)))


def tbe_grouped_linear_backward_weight(x: torch.Tensor, grad_y: torch.Tensor, offsets: torch.Tensor,
                                       grad_weight: torch.Tensor, grad_bias: Optional[torch.Tensor],
                                       workspace: Optional[torch.Tensor], stream=None):
    """grad_weight[e] = the sum of outer products of expert e's rows, grad_bias[e] their grad_y's sum."""
    experts, outer, inner = _grouped(grad_weight.shape, offsets)
    rows = x.shape[0]
    xs, gs = _rows("x", x, (rows, inner)), _rows("grad_y", grad_y, (rows, outer))
    _whole("grad_weight", grad_weight, grad_weight.shape)
    if grad_bias is not None:
        _whole("grad_bias", grad_bias, (experts, outer), grad_weight.dtype)
    _same([("x", x), ("grad_y", grad_y)])
    st = lib().tbe_grouped_linear_backward_weight(rows, experts, inner, outer, _ptr(x), xs, _ptr(grad_y), gs,
                                                  _dtype("x", x), _ptr(offsets), _I_DTYPE[offsets.dtype],
                                                  _ptr(grad_weight), _ptr(grad_bias),
                                                  _dtype("grad_weight", grad_weight), _ptr(workspace),
                                                  _bytes(workspace), _stream(stream))
    _check(st, "tbe_grouped_linear_backward_weight")


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
class AdamWTensors:
    """The tensors of a step, as an array of tbe_adamw_tensor on the host (the tensors are kept alive
    here).  States are float32, or uint8 codes with uint8 scales of ceil(numel / TBE_ADAMW_BLOCK)
    bytes; gradients are read from the same buffers at every step."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                 exp_avg: Sequence[torch.Tensor], exp_avg_sq: Sequence[torch.Tensor],
                 weight_decay: Union[float, Sequence[float]] = 0.0,
                 masters: Optional[Sequence[Optional[torch.Tensor]]] = None,
                 exp_avg_scales: Optional[Sequence[Optional[torch.Tensor]]] = None,
                 exp_avg_sq_scales: Optional[Sequence[Optional[torch.Tensor]]] = None):
        n = len(params)
        none = [None] * n
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else list(weight_decay)
        self.tensors = [list(x) if x is not None else none for x in
                        (params, grads, exp_avg, exp_avg_sq, masters, exp_avg_scales, exp_avg_sq_scales)]
        _need(all(len(x) == n for x in self.tensors) and len(decay) == n,
              f"{n} params need as many gradients, states and weight decays")
        self.c = (tbe_adamw_tensor * max(1, n))()
        self.count = n
        for i, (p, g, m, v, w, ms, vs) in enumerate(zip(*self.tensors)):
            numel = p.numel()
            eight = m.dtype == torch.uint8
            st = torch.uint8 if eight else torch.float32
            for name, t, size, dt in (("param", p, numel, None), ("gradient", g, numel, None),
                                      ("exp_avg", m, numel, st), ("exp_avg_sq", v, numel, st),
                                      ("master", w, numel, torch.float32),
                                      ("exp_avg_scale", ms, -(-numel // TBE_ADAMW_BLOCK), torch.uint8),
                                      ("exp_avg_sq_scale", vs, -(-numel // TBE_ADAMW_BLOCK), torch.uint8)):
                if t is None:
                    _need("scale" not in name or not eight, f"tensor {i}: states of 8 bits need scales")
                    continue
                _on_gpu(f"tensor {i}: {name}", t)
                _need(t.is_contiguous() and t.numel() == size and (dt is None or t.dtype == dt),
                      f"tensor {i}: {name} is {t.dtype} of {t.numel()} with strides {tuple(t.stride())}: "
                      f"contiguous {'' if dt is None else dt} of {size} is needed")
            self.c[i] = tbe_adamw_tensor(
                p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), None if w is None else w.data_ptr(),
                ms.data_ptr() if eight else None, vs.data_ptr() if eight else None, numel, decay[i],
                _dtype(f"tensor {i}: param", p), _dtype(f"tensor {i}: gradient", g),
                TBE_STATE_8BIT if eight else TBE_STATE_F32)


def tbe_adamw_step(tensors: AdamWTensors, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                   eps: float = 1e-8, control: Optional[torch.Tensor] = None, stream=None):
    """One AdamW step on every tensor.  control (float64, on the GPU): step, lr factor, gradient
    factor, skip; its step takes the place of `step`."""
    if control is not None:
        _whole("control", control, (TBE_ADAMW_CONTROL,), torch.float64)
    st = lib().tbe_adamw_step(tensors.c, tensors.count, int(step), float(lr), float(beta1), float(beta2),
                              float(eps), _ptr(control), _stream(stream))
    _check(st, "tbe_adamw_step")


def tbe_adamw_state_read(tensors: AdamWTensors, exp_avg_out: Sequence[torch.Tensor],
                         exp_avg_sq_out: Sequence[torch.Tensor], stream=None):
    """The values of states of 8 bits, into float32 or bfloat16 tensors (both hold them exactly)."""
    n = tensors.count
    _need(len(exp_avg_out) == n and len(exp_avg_sq_out) == n, f"{n} tensors need as many outputs of each state")
    outs = list(exp_avg_out) + list(exp_avg_sq_out)
    dtype = outs[0].dtype if outs else torch.float32
    for k, t in enumerate(outs):
        _on_gpu(f"output {k % n}", t)
        _need(t.is_contiguous() and t.numel() == tensors.c[k % n].numel and t.dtype == dtype,
              f"output {k % n} is {t.dtype} of {t.numel()}: contiguous {dtype} of {tensors.c[k % n].numel} is needed")
    array = ctypes.c_void_p * max(1, n)
    st = lib().tbe_adamw_state_read(tensors.c, n, array(*[t.data_ptr() for t in exp_avg_out]),
                                    array(*[t.data_ptr() for t in exp_avg_sq_out]),
                                    _dtype("outputs", outs[0]) if outs else 0, _stream(stream))
    _check(st, "tbe_adamw_state_read")
