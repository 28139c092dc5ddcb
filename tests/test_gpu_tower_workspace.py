"""The grouped weight gradient's workspace on the GPU: nothing behind it is written, and sums of shared rows are
right wherever their partial sums lie in it."""
import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print
from test_gpu_tower_grouped import Case

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def weight_gradient(c, bytes_):
    """The gradients, with a workspace of exactly these bytes and a guard behind it."""
    gw = torch.full((c.E, c.outer, c.inner), float("nan"), dtype=c.out, device="cuda")
    gb = torch.full((c.E, c.outer), float("nan"), dtype=c.out, device="cuda")
    buf = torch.full((bytes_ + 4096,), 255, dtype=torch.uint8, device="cuda")
    tbe.tbe_grouped_linear_backward_weight(c.x, c.gy, c.off, gw, gb, buf[:bytes_])
    torch.cuda.synchronize()
    assert (buf[bytes_:] == 255).all(), "wrote behind the workspace"
    for e, s in c.spans():
        g, x, n = c.gy[s].double(), c.x[s].double(), c.groups[e]
        c.check(f"grad_weight of expert {e}", gw[e], g.t() @ x, g.abs().t() @ x.abs(), n)
        c.check(f"grad_bias of expert {e}", gb[e], g.sum(0), g.abs().sum(0), n)


SKEWED = [9000, 300, 0, 4100, 200, 1900, 100]


@pytest.mark.parametrize("groups,inner,outer,dtype", [
    (SKEWED, 264, 136, BF16), (SKEWED, 1001, 75, F16), ([15600], 264, 136, BF16), ([0, 15600, 0], 264, 136, F16),
    ([1000] * 30 + [3, 0, 210], 264, 136, BF16),
    # several and single shares on both sides of the 64 experts that a wave counts at a time
    ([20000, 7, 0, 600] + [40] * 58 + [513, 512, 30000, 1, 0, 900, 2, 9500], 48, 40, BF16),
    ([1] * 66 + [39000, 30, 26000], 17, 9, F16),
])
def test_shared_rows_next_to_whole_experts(groups, inner, outer, dtype):
    flush_print("weight gradient", groups[:8], inner, outer)
    c = Case(groups, inner, outer, dtype, pad_rows=5)
    n = tbe.tbe_grouped_linear_backward_weight_workspace_bytes(c.rows, c.E, inner, outer)
    assert n > 0, "sizes whose rows are shared"
    weight_gradient(c, n)


def test_one_workspace_for_every_smaller_batch():
    """Sized for the largest batch, as a training program does."""
    inner, outer, largest = 520, 264, 20000
    for experts in (1, 4):
        n = tbe.tbe_grouped_linear_backward_weight_workspace_bytes(largest, experts, inner, outer)
        for rows in (largest, 19999, 13000, 8192, 4160, 4032, 1025, 513, 512, 40, 1):
            groups = [rows] if experts == 1 else [rows // 2, rows // 8, 0, rows - rows // 2 - rows // 8]
            flush_print("weight gradient", groups)
            weight_gradient(Case(groups, inner, outer, BF16), n)
