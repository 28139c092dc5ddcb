"""What the entry points of include/tbe_items.h refuse, on the host and before any launch, and the sizes of their
workspaces: no GPU needed."""
import ctypes

import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from bwd_tbe_fwd_amd import items

P = ctypes.c_void_p
A = P(4096)   # any address: the calls below must fail before it is used
OK, ARG, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BIG = 1 << 40


def error():
    return tbe.lib().tbe_last_error()


def lookup_forward(n=4, E=5, width=8, table=A, ts=8, tt=2, ids=A, it=0, scale=1.0, y=A, ys=8, yt=2):
    return tbe.lib().tbe_lookup_forward(n, E, width, table, ts, tt, ids, it, scale, y, ys, yt, None)


def test_lookup_forward_refusals():
    for kw, st, word in ((dict(n=-1), ARG, b"ids"), (dict(E=0), ARG, b"items"), (dict(width=0), ARG, b"width"),
                         (dict(n=1 << 31), UNSUPPORTED, b"ids"), (dict(E=(1 << 31) - 1), UNSUPPORTED, b"items"),
                         (dict(width=(1 << 20) + 1), UNSUPPORTED, b"width"), (dict(table=None), ARG, b"table is NULL"),
                         (dict(table=P(4097)), ARG, b"aligned"), (dict(tt=0, table=P(4098)), ARG, b"aligned"),
                         (dict(ts=7), ARG, b"apart"), (dict(ts=(1 << 31) + 1), ARG, b"apart"),
                         (dict(tt=3), UNSUPPORTED, b"type"), (dict(ids=None), ARG, b"ids"), (dict(it=2), ARG, b"type"),
                         (dict(it=1, ids=P(4100)), ARG, b"aligned"), (dict(y=None), ARG, b"y is NULL"),
                         (dict(ys=7), ARG, b"apart"), (dict(yt=-1), UNSUPPORTED, b"type")):
        assert lookup_forward(**kw) == st and word in error(), (kw, error())
    assert lookup_forward(n=0, ids=None, y=None) == OK and error() == b""


def lookup_backward(n=4, E=5, width=8, ids=A, it=0, gy=A, gs=8, yt=2, scale=1.0, gt=A, ts=8, tt=2, add=0, ws=A, nb=BIG):
    return tbe.lib().tbe_lookup_backward(n, E, width, ids, it, gy, gs, yt, scale, gt, ts, tt, add, ws, nb, None)


def test_lookup_backward_refusals():
    need = tbe.tbe_lookup_backward_workspace_bytes(4, 5, 8)
    assert need > 0
    for kw, st, word in ((dict(n=-1), ARG, b"ids"), (dict(E=0), ARG, b"items"), (dict(width=0), ARG, b"width"),
                         (dict(gy=None), ARG, b"grad_y"), (dict(gs=3), ARG, b"apart"), (dict(gt=None), ARG, b"grad_table"),
                         (dict(ts=3), ARG, b"apart"), (dict(yt=7), UNSUPPORTED, b"type"), (dict(tt=7), UNSUPPORTED, b"type"),
                         (dict(it=5), ARG, b"type"), (dict(ids=None), ARG, b"ids"), (dict(ws=None), WORKSPACE, b"workspace"),
                         (dict(ws=P(4096 + 64)), WORKSPACE, b"workspace"), (dict(nb=need - 1), WORKSPACE, b"workspace")):
        assert lookup_backward(**kw) == st and word in error(), (kw, error())
    assert lookup_backward(n=0, ids=None, gy=None, add=1) == OK and error() == b""


def test_lookup_workspace_serves_every_smaller_batch():
    for E, width in ((10, 8), (3001, 515), (131072, 1024), (2000000, 128)):
        last = 0
        for n in sorted({0, 1, 15, 16, 17, 63, 64, 65, 4095, 4096, 4097, 65535, 65536, 69631, 69632, 70000, 524287, 524288,
                         2048 * 4096 - 1, 2048 * 4096, 2048 * 4096 + 1, 1 << 23, (1 << 23) + 5, 1 << 24}):
            for m in (n, n + 1):
                need = tbe.tbe_lookup_backward_workspace_bytes(m, E, width)
                assert need >= last, (E, width, m)
                last = need
    assert tbe.tbe_lookup_backward_workspace_bytes(-1, 5, 8) == 0
    assert tbe.tbe_lookup_backward_workspace_bytes(4, 0, 8) == 0


def test_binding_checks_shapes_and_types(monkeypatch):
    """On tensors of the CPU, with the device check answered as if they lay on the current GPU."""
    monkeypatch.setattr(items, "_device", lambda: -1)
    monkeypatch.setattr(items, "_current", lambda stream, dev: None)
    t, ids, y = torch.zeros(5, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4, 8)
    ws = torch.zeros(256, dtype=torch.uint8)
    for call, word in ((lambda: tbe.tbe_lookup_forward(t, ids.float(), 1.0, y), "int32 or int64"),
                       (lambda: tbe.tbe_lookup_forward(t, ids[None], 1.0, y), "shape"),
                       (lambda: tbe.tbe_lookup_forward(t, torch.zeros(8, dtype=torch.int64)[::2], 1.0, y), "strides"),
                       (lambda: tbe.tbe_lookup_forward(t, ids, 1.0, y[:, :7]), "y has shape"),
                       (lambda: tbe.tbe_lookup_forward(t.t(), ids, 1.0, y), "contiguous"),
                       (lambda: tbe.tbe_lookup_forward(t.double(), ids, 1.0, y), "float32, float16 or bfloat16"),
                       (lambda: tbe.tbe_lookup_backward(ids, y[:3], 1.0, t, ws), "grad_y has shape"),
                       (lambda: tbe.tbe_lookup_backward(ids, y, 1.0, t.long(), ws), "float32, float16 or bfloat16"),
                       (lambda: tbe.tbe_lookup_backward(ids, y, 1.0, t, ws[:10]), "workspace")):
        with pytest.raises(tbe.TbeError, match=word):
            call()
    monkeypatch.setattr(items, "_device", lambda: 0)
    with pytest.raises(tbe.TbeError, match="not on the current GPU"):
        tbe.tbe_lookup_forward(t, ids, 1.0, y)


def loss_forward(rows=4, items=5, width=8, x=A, xs=8, w=A, ws=8, dt=2, b=A, t=A, tt=0, scale=1.0, loss=A, lse=A, work=A, nb=BIG):
    return tbe.lib().tbe_cross_entropy_forward(rows, items, width, x, xs, w, ws, dt, b, t, tt, scale, loss, lse, work, nb, None)


def loss_backward(rows=4, items=5, width=8, x=A, xs=8, w=A, ws=8, dt=2, b=A, t=A, tt=0, scale=1.0, lse=A, gl=A, gx=A, gxs=8, gw=A,
                  gws=8, gb=A, work=A, nb=BIG):
    return tbe.lib().tbe_cross_entropy_backward(rows, items, width, x, xs, w, ws, dt, b, t, tt, scale, lse, gl, gx, gxs, gw, gws, gb,
                                                work, nb, None)


COMMON = ((dict(rows=-1), ARG, b"rows"), (dict(items=0), ARG, b"items"), (dict(width=0), ARG, b"width"),
          (dict(rows=(1 << 22) + 1), UNSUPPORTED, b"rows"), (dict(items=(1 << 31) - 1), UNSUPPORTED, b"items"),
          (dict(width=(1 << 16) + 1), UNSUPPORTED, b"width"), (dict(dt=0), UNSUPPORTED, b"type"), (dict(dt=3), UNSUPPORTED, b"type"),
          (dict(scale=float("inf")), ARG, b"scale"), (dict(scale=float("nan")), ARG, b"scale"), (dict(x=None), ARG, b"x is NULL"),
          (dict(x=P(4097)), ARG, b"aligned"), (dict(xs=7), ARG, b"apart"), (dict(w=None), ARG, b"weight is NULL"),
          (dict(ws=7), ARG, b"apart"), (dict(ws=(1 << 31) + 1), ARG, b"apart"), (dict(b=P(4098)), ARG, b"bias"),
          (dict(t=None), ARG, b"targets"), (dict(tt=2), ARG, b"type"), (dict(tt=1, t=P(4100)), ARG, b"aligned"),
          (dict(lse=None), ARG, b"lse"), (dict(lse=P(4098)), ARG, b"lse"), (dict(work=None), WORKSPACE, b"workspace"),
          (dict(work=P(4096 + 128)), WORKSPACE, b"workspace"))


def test_cross_entropy_refusals():
    need = tbe.tbe_cross_entropy_forward_workspace_bytes(4, 5, 8)
    for kw, st, word in COMMON + ((dict(loss=None), ARG, b"loss"), (dict(nb=need - 1), WORKSPACE, b"workspace")):
        assert loss_forward(**kw) == st and word in error(), (kw, error())
    assert loss_forward(rows=0, x=None, t=None, loss=None, lse=None, work=None) == OK and error() == b""
    need = tbe.tbe_cross_entropy_backward_workspace_bytes(4, 5, 8)
    for kw, st, word in COMMON + ((dict(gl=None), ARG, b"grad_loss"), (dict(gxs=7), ARG, b"grad_x"), (dict(gx=P(4097)), ARG, b"grad_x"),
                                  (dict(gws=7), ARG, b"grad_weight"), (dict(gb=P(4098)), ARG, b"grad_bias"),
                                  (dict(nb=need - 1), WORKSPACE, b"workspace")):
        assert loss_backward(**kw) == st and word in error(), (kw, error())
    assert loss_backward(gx=None, gw=None, gb=None) == OK and error() == b""


def test_cross_entropy_workspaces_serve_every_smaller_batch():
    sizes = sorted({1, 2, 7, 63, 64, 65, 255, 256, 257, 511, 512, 513, 1000, 1023, 1024, 1025, 2048, 4095, 4096, 8191, 8192, 8193, 32767,
                    65536, 131071, 131072, 131073, 500000, 1 << 20, 1 << 22})
    for of in (tbe.tbe_cross_entropy_forward_workspace_bytes, tbe.tbe_cross_entropy_backward_workspace_bytes):
        for items, width in ((1, 1), (5, 8), (3001, 515), (131072, 1024), (2000000, 128), ((1 << 31) - 2, 4)):
            last = 0
            for n in sizes:
                need = of(n, items, width)
                assert need >= last, (items, width, n)
                last = need
        assert of(-1, 5, 8) == 0 and of(4, 0, 8) == 0
    # a training batch's logits would take 8192 x 131072 x 2 bytes = 2 GiB in 16 bits
    assert tbe.tbe_cross_entropy_forward_workspace_bytes(8192, 131072, 1024) < 128 << 20
    assert tbe.tbe_cross_entropy_backward_workspace_bytes(8192, 131072, 1024) < 768 << 20


def test_loss_binding_checks_shapes_and_types(monkeypatch):
    monkeypatch.setattr(items, "_device", lambda: -1)
    monkeypatch.setattr(items, "_current", lambda stream, dev: None)
    h = torch.bfloat16
    x, w, t, v = torch.zeros(4, 8, dtype=h), torch.zeros(5, 8, dtype=h), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    b, ws = torch.zeros(5), torch.zeros(256, dtype=torch.uint8)

    def forward(x=x, w=w, b=b, t=t, loss=v, lse=v, ws=ws):
        tbe.tbe_cross_entropy_forward(x, w, b, t, 1.0, loss, lse, ws)

    def backward(lse=v, gl=v, gx=x, gw=w, gb=b):
        tbe.tbe_cross_entropy_backward(x, w, b, t, 1.0, lse, gl, gx, gw, gb, ws)

    for call, word in ((lambda: forward(x=x[:, :7]), "rows of 7"), (lambda: forward(w=w.half()), "not of x's type"),
                       (lambda: forward(b=b.double()), "bias is"), (lambda: forward(b=torch.zeros(4)), "bias has shape"),
                       (lambda: forward(t=t[:3]), "targets have shape"), (lambda: forward(t=t.float()), "int32 or int64"),
                       (lambda: forward(loss=v[:3]), "loss has shape"), (lambda: forward(lse=v.half()), "lse is"),
                       (lambda: forward(x=x.float(), w=w.float()), "fp16 or bf16"), (lambda: forward(ws=ws[:8]), "workspace"),
                       (lambda: backward(gl=v.half()), "grad_loss is"), (lambda: backward(gx=x.float()), "grad_x is not"),
                       (lambda: backward(gx=x[:3]), "grad_x has shape"), (lambda: backward(gw=w.t()), "grad_weight has shape"),
                       (lambda: backward(gw=w.half()), "grad_weight is not"), (lambda: backward(gb=torch.zeros(4)), "grad_bias has shape")):
        with pytest.raises(tbe.TbeError, match=word):
            call()


def test_cross_entropy_scales():
    need = tbe.tbe_cross_entropy_forward_workspace_bytes(4, 5, 8)
    for scale in (2.0 ** -65, -2.0 ** -100, 1e-40, 2.0 ** 65, -3e38):
        assert loss_forward(scale=scale) == UNSUPPORTED and b"scale" in error()
        assert loss_backward(scale=scale) == UNSUPPORTED and b"scale" in error()
    for scale in (0.0, 2.0 ** -64, -2.0 ** 64):  # what comes after the scale is looked at
        assert loss_forward(scale=scale, nb=need - 1) == WORKSPACE
