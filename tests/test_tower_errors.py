"""The error text of the tower's entry points, and what the binding refuses before a call.  No GPU needed."""
import ctypes

import pytest

import bwd_tbe_fwd_amd as tbe
from bwd_tbe_fwd_amd import tower

P = ctypes.c_void_p
A = P(4096)


def test_a_call_that_succeeds_leaves_no_error_text():
    L = tbe.lib()
    none = (tbe.tbe_adamw_tensor * 1)()
    calls = (lambda: L.tbe_layer_norm_forward(0, 8, None, 8, 0, None, None, 0, 1e-5, None, 8, 0, None, None, None),
             lambda: L.tbe_layer_norm_backward(0, 8, None, 8, 0, None, 8, 0, None, None, None, 0, None, 8, None, None, None, 0, None),
             lambda: L.tbe_grouped_linear_forward(0, 2, 8, 8, None, 8, A, None, 2, A, 0, None, 8, 2, None),
             lambda: L.tbe_grouped_linear_backward_input(0, 2, 8, 8, None, 8, A, 2, A, 0, None, 8, 2, None),
             lambda: L.tbe_adamw_step(none, 1, 1, 1e-3, 0.9, 0.999, 1e-8, None, None),
             lambda: L.tbe_adamw_state_read(none, 0, None, None, 0, None))
    for call in calls:
        assert L.tbe_adamw_step(None, -1, 1, 1e-3, 0.9, 0.999, 1e-8, None, None) == 1
        assert L.tbe_last_error() != b""
        assert call() == 0
        assert L.tbe_last_error() == b""


def test_steps_are_taken_on_the_tensors_gpu(monkeypatch):
    """A plan made on one GPU is refused where another one is current: its kernels would run there."""
    monkeypatch.setattr(tower, "_device", lambda: 0)
    monkeypatch.setattr(tower, "_current", lambda stream, dev: None)
    plan = tbe.AdamWTensors([], [], [], [])
    tbe.tbe_adamw_step(plan, 1, 1e-3)
    tbe.tbe_adamw_state_read(plan, [], [])
    monkeypatch.setattr(tower, "_device", lambda: 1)
    for call in (lambda: tbe.tbe_adamw_step(plan, 1, 1e-3), lambda: tbe.tbe_adamw_state_read(plan, [], [])):
        with pytest.raises(tbe.TbeError, match="GPU 0"):
            call()
