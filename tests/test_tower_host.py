"""What the dense tower's entry points refuse, on the host and before any launch: no GPU needed."""
import ctypes
import subprocess

import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from test_abi import ROOT

P = ctypes.c_void_p
A = P(4096)   # any address: the calls below must fail before it is used
OK, ARG, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def error():
    return tbe.lib().tbe_last_error()


def norm_forward(rows=4, width=8, x=A, xs=8, xt=0, w=A, b=A, wt=0, eps=1e-5, y=A, ys=8, yt=0, mean=A, rstd=A):
    return tbe.lib().tbe_layer_norm_forward(rows, width, x, xs, xt, w, b, wt, eps, y, ys, yt, mean, rstd, None)


def test_norm_forward_refusals():
    for kw, st, word in ((dict(rows=-1), ARG, b"rows"), (dict(width=0), ARG, b"rows"),
                         (dict(width=(1 << 24) + 1), UNSUPPORTED, b"width"), (dict(rows=1 << 31), UNSUPPORTED, b"rows"),
                         (dict(x=None), ARG, b"x is NULL"), (dict(y=None), ARG, b"y is NULL"),
                         (dict(x=P(4098)), ARG, b"aligned"), (dict(xt=1, x=P(4097)), ARG, b"aligned"),
                         (dict(xs=7), ARG, b"apart"), (dict(ys=7), ARG, b"apart"), (dict(xt=3), UNSUPPORTED, b"type"),
                         (dict(yt=-1), UNSUPPORTED, b"type"), (dict(wt=9), UNSUPPORTED, b"type"),
                         (dict(w=P(4097), wt=2), ARG, b"aligned"), (dict(eps=-1.0), ARG, b"eps"),
                         (dict(eps=float("nan")), ARG, b"eps"), (dict(mean=P(4098)), ARG, b"mean")):
        assert norm_forward(**kw) == st and word in error(), (kw, error())
    assert norm_forward(rows=0, x=None, y=None) == OK


def norm_backward(rows=4, width=8, x=A, xs=8, xt=0, gy=A, gs=8, yt=0, mean=A, rstd=A, w=A, wt=0, gx=A, os=8, gw=A, gb=A,
                  ws=A, n=1 << 20):
    return tbe.lib().tbe_layer_norm_backward(rows, width, x, xs, xt, gy, gs, yt, mean, rstd, w, wt, gx, os, gw, gb, ws, n, None)


def test_norm_backward_refusals():
    need = tbe.tbe_layer_norm_backward_workspace_bytes(4, 8)
    assert need == 4 * 2 * 8 * 4
    for kw, st, word in ((dict(rows=-1), ARG, b"rows"), (dict(gy=None), ARG, b"grad_y"), (dict(gs=3), ARG, b"apart"),
                         (dict(os=3), ARG, b"grad_x"), (dict(mean=None), ARG, b"mean"), (dict(rstd=None), ARG, b"mean"),
                         (dict(ws=None), WORKSPACE, b"workspace"), (dict(n=need - 1), WORKSPACE, b"workspace"),
                         (dict(ws=P(4096 + 16)), WORKSPACE, b"workspace"), (dict(wt=5), UNSUPPORTED, b"type")):
        assert norm_backward(**kw) == st and word in error(), (kw, error())


def test_norm_workspace_stays_small():
    assert tbe.tbe_layer_norm_backward_workspace_bytes(10 ** 6, 4096) == 1024 * 2 * 4096 * 4
    # wide rows take fewer partial rows: 32 MiB of each sum, or 8 rows
    assert tbe.tbe_layer_norm_backward_workspace_bytes(10 ** 6, 1 << 17) == 64 * 2 * (1 << 17) * 4
    assert tbe.tbe_layer_norm_backward_workspace_bytes(10 ** 6, 1 << 24) == 8 * 2 * (1 << 24) * 4
    assert tbe.tbe_layer_norm_backward_workspace_bytes(-1, 8) == 0


def grouped_forward(rows=4, E=2, inner=8, outer=8, x=A, xs=8, w=A, b=A, dt=2, off=A, ot=0, y=A, ys=8, od=2):
    return tbe.lib().tbe_grouped_linear_forward(rows, E, inner, outer, x, xs, w, b, dt, off, ot, y, ys, od, None)


def test_grouped_refusals():
    L = tbe.lib()
    cases = ((dict(rows=-1), ARG, b"rows"), (dict(E=0), ARG, b"experts"), (dict(inner=0), ARG, b"inner"),
             (dict(outer=0), ARG, b"outer"), (dict(rows=(1 << 29) + 1), UNSUPPORTED, b"more than"),
             (dict(E=65536), UNSUPPORTED, b"more than"), (dict(inner=(1 << 20) + 1), UNSUPPORTED, b"more than"),
             (dict(dt=0, od=0), UNSUPPORTED, b"types"), (dict(dt=2, od=1), UNSUPPORTED, b"types"),
             (dict(dt=7), UNSUPPORTED, b"types"), (dict(ot=2), ARG, b"offset type"), (dict(off=None), ARG, b"offsets"),
             (dict(off=P(4100), ot=1), ARG, b"offsets"), (dict(x=None), ARG, b"x is NULL"),
             (dict(x=P(4097)), ARG, b"aligned"), (dict(w=None), ARG, b"weight"), (dict(b=P(4097)), ARG, b"bias"),
             (dict(y=None), ARG, b"y is NULL"), (dict(xs=7), ARG, b"apart"), (dict(ys=7), ARG, b"apart"),
             (dict(od=0, y=P(4098)), ARG, b"aligned"))
    for kw, st, word in cases:
        assert grouped_forward(**kw) == st and word in error(), (kw, error())
    assert grouped_forward(rows=0, x=None, y=None) == OK

    def inp(gy=A, gs=8, w=A, off=A, gx=A, xs=8, dt=2, od=2):
        return L.tbe_grouped_linear_backward_input(4, 2, 8, 8, gy, gs, w, dt, off, 0, gx, xs, od, None)

    for kw, word in ((dict(gy=None), b"grad_y"), (dict(gs=1), b"apart"), (dict(w=None), b"weight"), (dict(off=None), b"offsets"),
                     (dict(gx=None), b"grad_x"), (dict(xs=1), b"apart")):
        assert inp(**kw) == ARG and word in error(), (kw, error())

    # sizes whose weights' gradient needs a workspace, if any does
    need = tbe.tbe_grouped_linear_backward_weight_workspace_bytes(1 << 20, 1, 64, 64)

    def wgt(x=A, xs=64, gy=A, gs=64, gw=A, gb=A, dt=2, od=0, ws=A, n=need):
        return L.tbe_grouped_linear_backward_weight(1 << 20, 1, 64, 64, x, xs, gy, gs, dt, A, 0, gw, gb, od, ws, n, None)

    for kw, word in ((dict(x=None), b"x is NULL"), (dict(gy=None), b"grad_y"), (dict(xs=1), b"apart"), (dict(gs=1), b"apart"),
                     (dict(gw=None), b"grad_weight"), (dict(gb=P(4098)), b"grad_bias")):
        assert wgt(**kw) == ARG and word in error(), (kw, error())
    if need:
        for kw in (dict(ws=None), dict(n=need - 1), dict(ws=P(4096 + 8))):
            assert wgt(**kw) == WORKSPACE and b"workspace" in error()


def adamw(n=1, step=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, control=None, count=1, null=False, **fields):
    t = (tbe.tbe_adamw_tensor * 1)()
    base = dict(param=4096, grad=4096, exp_avg=4096, exp_avg_sq=4096, numel=n, param_dtype=0, grad_dtype=0, state=0)
    for k, v in {**base, **fields}.items():
        setattr(t[0], k, v)
    return tbe.lib().tbe_adamw_step(None if null else t, count, step, lr, b1, b2, eps, control, None)


def test_adamw_refusals():
    for kw, st, word in ((dict(count=-1), ARG, b"tensors"), (dict(null=True), ARG, b"tensors"), (dict(step=0), ARG, b"step"),
                         (dict(b1=1.0), ARG, b"beta1"), (dict(b2=-0.1), ARG, b"beta2"), (dict(eps=-1.0), ARG, b"eps"),
                         (dict(lr=float("inf")), ARG, b"lr"), (dict(control=P(4100)), ARG, b"control"),
                         (dict(param_dtype=4), UNSUPPORTED, b"type"), (dict(grad_dtype=-1), UNSUPPORTED, b"type"),
                         (dict(state=2), UNSUPPORTED, b"state"), (dict(master=4096), UNSUPPORTED, b"master"),
                         (dict(n=-1), ARG, b"numel"), (dict(n=(1 << 34) + 1), ARG, b"numel"), (dict(param=None), ARG, b"NULL"),
                         (dict(grad=None), ARG, b"NULL"), (dict(exp_avg=None), ARG, b"NULL"), (dict(exp_avg_sq=None), ARG, b"NULL"),
                         (dict(state=1), ARG, b"NULL"), (dict(param=4098), ARG, b"aligned"), (dict(exp_avg=4097), ARG, b"aligned"),
                         (dict(grad=4097, grad_dtype=2), ARG, b"aligned")):
        assert adamw(**kw) == st and word in error(), (kw, error())
    assert adamw(count=0, null=True) == OK
    assert adamw(n=0, param=None, grad=None) == OK

    L = tbe.lib()
    t = (tbe.tbe_adamw_tensor * 1)()
    outs = (ctypes.c_void_p * 1)(4096)
    t[0].numel, t[0].param, t[0].grad, t[0].exp_avg, t[0].exp_avg_sq = 8, 4096, 4096, 4096, 4096
    assert L.tbe_adamw_state_read(t, 1, outs, outs, 0, None) == ARG and b"32 bits" in error()
    t[0].state, t[0].exp_avg_scale, t[0].exp_avg_sq_scale = 1, 4096, 4096
    assert L.tbe_adamw_state_read(t, 1, outs, outs, 1, None) == UNSUPPORTED and b"exact" in error()
    assert L.tbe_adamw_state_read(t, 1, outs, None, 0, None) == ARG
    assert L.tbe_adamw_state_read(t, 1, outs, (ctypes.c_void_p * 1)(), 0, None) == ARG and b"output" in error()


def test_adamw_struct_layout(tmp_path):
    src = tmp_path / "layout.c"
    fields = [f for f, _ in tbe.tbe_adamw_tensor._fields_]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "%s/include/tbe_tower.h"\nint main(void) {\n' % ROOT +
                   "".join('  printf("%%zu ", offsetof(tbe_adamw_tensor, %s));\n' % f for f in fields) +
                   '  printf("%zu %d %d %d", sizeof(tbe_adamw_tensor), TBE_ADAMW_BLOCK, TBE_ADAMW_CONTROL, '
                   'TBE_LAYER_NORM_MAX_WIDTH);\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-o", str(exe), str(src)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert got == [getattr(tbe.tbe_adamw_tensor, f).offset for f in fields] + [
        ctypes.sizeof(tbe.tbe_adamw_tensor), tbe.TBE_ADAMW_BLOCK, tbe.TBE_ADAMW_CONTROL, tbe.TBE_LAYER_NORM_MAX_WIDTH]


@pytest.mark.skipif(torch.cuda.is_available(), reason="tensors of the CPU, as a caller without a GPU would pass them")
def test_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(4, 8)
    with pytest.raises(tbe.TbeError, match="not on the current GPU"):
        tbe.tbe_layer_norm_forward(x, None, None, 1e-5, x)
    with pytest.raises(tbe.TbeError, match="not on the current GPU"):
        tbe.tbe_grouped_linear_forward(x, torch.zeros(1, 8, 8), None, torch.zeros(2, dtype=torch.int32), x)
    with pytest.raises(tbe.TbeError, match="not on the current GPU"):
        tbe.AdamWTensors([x], [x], [x], [x])


@pytest.mark.gpu
def test_binding_refuses_shapes_and_types():
    x, bad = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 9, device="cuda")
    v = torch.zeros(8, device="cuda")
    for call, word in ((lambda: tbe.tbe_layer_norm_forward(x, None, None, 1e-5, bad), "shape"),
                       (lambda: tbe.tbe_layer_norm_forward(x.t(), None, None, 1e-5, x.t()), "contiguous"),
                       (lambda: tbe.tbe_layer_norm_forward(x, v[:7], None, 1e-5, x), "shape"),
                       (lambda: tbe.tbe_layer_norm_forward(x, v, v.half(), 1e-5, x), "float16"),
                       (lambda: tbe.tbe_layer_norm_forward(x.double(), None, None, 1e-5, x), "float64"),
                       (lambda: tbe.tbe_layer_norm_forward(x, None, None, 1e-5, x, v[:4].half()), "mean"),
                       (lambda: tbe.tbe_layer_norm_backward(x, x, v[:4], v[:4], None, x.half(), None, None, None), "grad_x"),
                       (lambda: tbe.tbe_layer_norm_backward(x, x, v[:4], v[:4], None, x, v, None, None), "workspace")):
        with pytest.raises(tbe.TbeError, match=word):
            call()
    xb, w = x.bfloat16(), torch.zeros(2, 5, 8, dtype=torch.bfloat16, device="cuda")
    off, y = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, 5, dtype=torch.bfloat16, device="cuda")
    for call, word in ((lambda: tbe.tbe_grouped_linear_forward(x, w, None, off, y), "type"),
                       (lambda: tbe.tbe_grouped_linear_forward(xb, w, None, off[:2], y), "offsets"),
                       (lambda: tbe.tbe_grouped_linear_forward(xb, w, None, off.float(), y), "offsets"),
                       (lambda: tbe.tbe_grouped_linear_forward(xb, w.transpose(1, 2), None, off, y), "shape"),
                       (lambda: tbe.tbe_grouped_linear_forward(xb, w, y, off, y), "bias"),
                       (lambda: tbe.tbe_grouped_linear_forward(xb, w, None, off, y[:, :4]), "shape"),
                       (lambda: tbe.tbe_grouped_linear_forward(xb, w, None, off, y.half()), "types"),
                       (lambda: tbe.tbe_grouped_linear_backward_input(y, w, off, xb[:, :7]), "shape"),
                       (lambda: tbe.tbe_grouped_linear_backward_weight(xb, y[:3], off, w, None, None), "shape"),
                       (lambda: tbe.tbe_grouped_linear_backward_weight(xb, y, off, w, y, None), "grad_bias")):
        with pytest.raises(tbe.TbeError, match=word):
            call()
    c, s = torch.zeros(8, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.uint8, device="cuda")
    for call, word in ((lambda: tbe.AdamWTensors([v], [v], [v], []), "as many"),
                       (lambda: tbe.AdamWTensors([v], [v[:7]], [v], [v]), "gradient"),
                       (lambda: tbe.AdamWTensors([v], [v], [v.half()], [v]), "exp_avg"),
                       (lambda: tbe.AdamWTensors([v], [v], [c], [c]), "scales"),
                       (lambda: tbe.AdamWTensors([v], [v], [c], [v], exp_avg_scales=[s], exp_avg_sq_scales=[s]), "exp_avg_sq"),
                       (lambda: tbe.AdamWTensors([v], [v], [c], [c], exp_avg_scales=[c], exp_avg_sq_scales=[s]), "exp_avg_scale"),
                       (lambda: tbe.AdamWTensors([v[::2]], [v[::2]], [v[:4]], [v[:4]]), "param"),
                       (lambda: tbe.AdamWTensors([v], [v], [v], [v], masters=[v]) and tbe.tbe_adamw_step(
                           tbe.AdamWTensors([v], [v], [v], [v], masters=[v]), 1, 1e-3), "master"),
                       (lambda: tbe.tbe_adamw_step(tbe.AdamWTensors([v], [v], [v], [v]), 1, 1e-3, control=v), "control"),
                       (lambda: tbe.tbe_adamw_state_read(tbe.AdamWTensors([v], [v], [v], [v]), [v], [v]), "32 bits")):
        with pytest.raises(tbe.TbeError, match=word):
            call()
