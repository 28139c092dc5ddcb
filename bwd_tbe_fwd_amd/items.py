"""The two ends of a model that reads and predicts the rows of one table (``include/tbe_items.h``): scaled
lookup of single rows with the table's dense gradient, softmax cross entropy over all rows with its gradients.

Argument marshalling as in tower.py: torch tensors in, the C entry point of the same name called on the
current stream, TbeError where it refuses.  What the C interface cannot see, a tensor's shape, strides,
type and device, is checked here.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _I_DTYPE, _check, lib
from .tower import _at, _bytes, _current, _device, _dtype, _off_gpu, _refuse, _rows, _same, _whole

TBE_ITEMS_MAX_WIDTH = 1 << 20
TBE_CROSS_ENTROPY_MAX_ROWS = 1 << 22
TBE_CROSS_ENTROPY_MAX_WIDTH = 1 << 16


def _ids(name: str, t: torch.Tensor, dev: int, n: Optional[int] = None) -> int:
    """The type of a contiguous vector of ids."""
    if t.get_device() != dev:
        _off_gpu(name, t)
    it = _I_DTYPE.get(t.dtype)
    if it is None:
        _refuse(f"{name} are {t.dtype}: int32 or int64 are supported")
    if t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        _refuse(f"{name} have shape {tuple(t.shape)} and strides {tuple(t.stride())}: contiguous "
                f"{'(n,)' if n is None else (n,)} is needed")
    return it


# ---------------------------------------------------------------------------
# lookup
# ---------------------------------------------------------------------------
def tbe_lookup_forward(table: torch.Tensor, ids: torch.Tensor, scale: float, y: torch.Tensor, stream=None):
    """y[i] = scale * table[ids[i]]; zero for an id outside the table."""
    dev = _device()
    ts = _rows("table", table, dev)
    items, width = table.shape
    it = _ids("ids", ids, dev)
    n = ids.shape[0]
    ys = _rows("y", y, dev, (n, width))
    st = lib().tbe_lookup_forward(n, items, width, table.data_ptr(), ts, _dtype("table", table), ids.data_ptr(), it, scale,
                                  y.data_ptr(), ys, _dtype("y", y), _current(stream, dev))
    _check(st, "tbe_lookup_forward")


def tbe_lookup_backward_workspace_bytes(num_ids: int, items: int, width: int) -> int:
    return int(lib().tbe_lookup_backward_workspace_bytes(int(num_ids), int(items), int(width)))


def tbe_lookup_backward(ids: torch.Tensor, grad_y: torch.Tensor, scale: float, grad_table: torch.Tensor,
                        workspace: Optional[torch.Tensor], accumulate: bool = False, stream=None):
    """grad_table[v] = scale * the sum of grad_y[i] over ids[i] = v, or (accumulate) has it added."""
    dev = _device()
    ts = _rows("grad_table", grad_table, dev)
    items, width = grad_table.shape
    it = _ids("ids", ids, dev)
    n = ids.shape[0]
    gs = _rows("grad_y", grad_y, dev, (n, width))
    st = lib().tbe_lookup_backward(n, items, width, ids.data_ptr(), it, grad_y.data_ptr(), gs, _dtype("grad_y", grad_y), scale,
                                   grad_table.data_ptr(), ts, _dtype("grad_table", grad_table), int(bool(accumulate)),
                                   _at(workspace), _bytes(workspace, dev), _current(stream, dev))
    _check(st, "tbe_lookup_backward")


# ---------------------------------------------------------------------------
# softmax cross entropy over all items
# ---------------------------------------------------------------------------
def tbe_cross_entropy_forward_workspace_bytes(rows: int, items: int, width: int) -> int:
    return int(lib().tbe_cross_entropy_forward_workspace_bytes(int(rows), int(items), int(width)))


def _loss_inputs(x, weight, bias, targets, dev):
    xs = _rows("x", x, dev)
    rows, width = x.shape
    ws = _rows("weight", weight, dev)
    items = weight.shape[0]
    if weight.shape[1] != width:
        _refuse(f"weight has shape {tuple(weight.shape)}, x rows of {width}")
    _same("weight", weight, "x", x.dtype)
    if bias is not None:
        _whole("bias", bias, dev, (items,), torch.float32)
    return rows, items, width, xs, ws, _ids("targets", targets, dev, rows)


def tbe_cross_entropy_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor], targets: torch.Tensor,
                              scale: float, loss: torch.Tensor, lse: torch.Tensor, workspace: Optional[torch.Tensor],
                              stream=None):
    """With logits = scale * x @ weight.T + bias: lse[i] = logsumexp(logits[i]), loss[i] = lse[i] -
    logits[i, targets[i]]; both 0 for a row whose target lies outside the items."""
    dev = _device()
    rows, items, width, xs, ws, tt = _loss_inputs(x, weight, bias, targets, dev)
    _whole("loss", loss, dev, (rows,), torch.float32)
    _whole("lse", lse, dev, (rows,), torch.float32)
    st = lib().tbe_cross_entropy_forward(rows, items, width, x.data_ptr(), xs, weight.data_ptr(), ws, _dtype("x", x), _at(bias),
                                         targets.data_ptr(), tt, scale, loss.data_ptr(), lse.data_ptr(), _at(workspace),
                                         _bytes(workspace, dev), _current(stream, dev))
    _check(st, "tbe_cross_entropy_forward")


def tbe_cross_entropy_backward_workspace_bytes(rows: int, items: int, width: int) -> int:
    return int(lib().tbe_cross_entropy_backward_workspace_bytes(int(rows), int(items), int(width)))


def tbe_cross_entropy_backward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor], targets: torch.Tensor,
                               scale: float, lse: torch.Tensor, grad_loss: torch.Tensor, grad_x: Optional[torch.Tensor],
                               grad_weight: Optional[torch.Tensor], grad_bias: Optional[torch.Tensor],
                               workspace: Optional[torch.Tensor], stream=None):
    """The gradients of tbe_cross_entropy_forward's losses, each weighted by grad_loss [rows]; any of the three may be
    left out (None)."""
    dev = _device()
    rows, items, width, xs, ws, tt = _loss_inputs(x, weight, bias, targets, dev)
    _whole("lse", lse, dev, (rows,), torch.float32)
    _whole("grad_loss", grad_loss, dev, (rows,), torch.float32)
    gxs = gws = 0
    if grad_x is not None:
        gxs = _rows("grad_x", grad_x, dev, x.shape)
        _same("grad_x", grad_x, "x", x.dtype)
    if grad_weight is not None:
        gws = _rows("grad_weight", grad_weight, dev, weight.shape)
        _same("grad_weight", grad_weight, "x", x.dtype)
    if grad_bias is not None:
        _whole("grad_bias", grad_bias, dev, (items,), torch.float32)
    st = lib().tbe_cross_entropy_backward(rows, items, width, x.data_ptr(), xs, weight.data_ptr(), ws, _dtype("x", x), _at(bias),
                                          targets.data_ptr(), tt, scale, lse.data_ptr(), grad_loss.data_ptr(), _at(grad_x), gxs,
                                          _at(grad_weight), gws, _at(grad_bias), _at(workspace), _bytes(workspace, dev),
                                          _current(stream, dev))
    _check(st, "tbe_cross_entropy_backward")
