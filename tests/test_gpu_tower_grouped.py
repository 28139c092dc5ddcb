"""Linear layers on rows grouped by expert, on the GPU against their definition in 64 bits.

Tolerance: products of 16-bit values are exact in fp32; a sum of K of them runs through the matrix
instructions, 32 or fewer terms each, so its depth is at most K / 8 + 32 roundings of at most 2 u
(u = 2^-24) of the sum of |terms|; the stored result adds its type's unit roundoff."""
import pytest
import torch

import bwd_tbe_fwd_amd as tbe
from gpu_util import flush_print
from test_gpu_tower_norm import LEAST, U, UNIT, check

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def draw(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def strided(shape, dtype, seed, pad, scale=1.0):
    """A matrix whose rows lie `pad` further apart, with NaN between them."""
    buf = torch.full((shape[0], shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :shape[1]] = draw(shape, dtype, seed, scale)
    return buf[:, :shape[1]]


class Case:
    def __init__(self, groups, inner, outer, dtype, pad_rows=0, pad=0, otype=torch.int32, out=None, bias=True, seed=1):
        self.groups, self.inner, self.outer, self.pad = groups, inner, outer, pad
        self.rows, self.E = sum(groups) + pad_rows, len(groups)
        self.used = sum(groups)
        self.off = torch.tensor([sum(groups[:i]) for i in range(self.E + 1)], dtype=otype, device="cuda")
        self.x = strided((self.rows, inner), dtype, seed, pad)
        self.gy = strided((self.rows, outer), dtype, seed + 1, pad, 0.1)
        if pad_rows:  # rows of no expert count for nothing, whatever they hold
            self.x[self.used:] = float("nan")
            self.gy[self.used:] = float("inf")
        self.w = draw((self.E, outer, inner), dtype, seed + 2, inner ** -0.5)
        self.b = draw((self.E, outer), dtype, seed + 3) if bias else None
        self.out = out or dtype

    def spans(self):
        at = 0
        for e, n in enumerate(self.groups):
            yield e, slice(at, at + n)
            at += n

    def empty(self, width):
        return torch.full((self.rows, width + 4), float("nan"), dtype=self.out, device="cuda")

    def check(self, what, got, exp, terms, depth):
        t = got.dtype
        check(what, got, exp, UNIT[t] * exp.abs() + LEAST[t] + 2 * U * (depth / 8 + 32) * terms)

    def forward(self):
        buf = self.empty(self.outer)
        y = buf[:, :self.outer]
        tbe.tbe_grouped_linear_forward(self.x, self.w, self.b, self.off, y)
        torch.cuda.synchronize()
        assert buf[:, self.outer:].isnan().all()
        assert not y[self.used:].any(), "rows of no expert are zero"
        for e, s in self.spans():
            b = 0.0 if self.b is None else self.b[e].double()
            x, w = self.x[s].double(), self.w[e].double()
            self.check(f"y of expert {e}", y[s], x @ w.t() + b, x.abs() @ w.abs().t() + abs(b), self.inner)
        return y.clone()

    def backward_input(self):
        buf = self.empty(self.inner)
        gx = buf[:, :self.inner]
        tbe.tbe_grouped_linear_backward_input(self.gy, self.w, self.off, gx)
        torch.cuda.synchronize()
        assert buf[:, self.inner:].isnan().all()
        assert not gx[self.used:].any(), "rows of no expert are zero"
        for e, s in self.spans():
            g, w = self.gy[s].double(), self.w[e].double()
            self.check(f"grad_x of expert {e}", gx[s], g @ w, g.abs() @ w.abs(), self.outer)
        return gx.clone()

    def backward_weight(self, bias=True):
        gw = torch.full((self.E, self.outer, self.inner), float("nan"), dtype=self.out, device="cuda")
        gb = torch.full((self.E, self.outer), float("nan"), dtype=self.out, device="cuda") if bias else None
        n = tbe.tbe_grouped_linear_backward_weight_workspace_bytes(self.rows, self.E, self.inner, self.outer)
        ws = tbe.workspace(n)
        ws.fill_(255)
        tbe.tbe_grouped_linear_backward_weight(self.x, self.gy, self.off, gw, gb, ws)
        torch.cuda.synchronize()
        for e, s in self.spans():
            g, x = self.gy[s].double(), self.x[s].double()
            n = self.groups[e]
            self.check(f"grad_weight of expert {e}", gw[e], g.t() @ x, g.abs().t() @ x.abs(), n)
            if bias:
                self.check(f"grad_bias of expert {e}", gb[e], g.sum(0), g.abs().sum(0), n)
            if n == 0:
                assert not gw[e].any() and (gb is None or not gb[e].any())
        return gw, gb

    def all(self):
        self.forward()
        self.backward_input()
        self.backward_weight()


# groups of no row, of one, of tiles' sizes and one to each side; sides of one, odd, whole tiles
GROUPS = {"one expert": [70], "one row each": [1, 1, 1], "empty first and last": [0, 33, 0, 64, 0],
          "around tiles": [63, 64, 65, 127, 128, 129, 31, 16, 17], "skewed": [700, 3, 0, 41, 256, 2]}


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("inner,outer", [(64, 64), (128, 256), (72, 40), (33, 1), (1, 65), (200, 129)])
def test_products(dtype, groups, inner, outer):
    flush_print("grouped", dtype, groups, inner, outer)
    Case(GROUPS[groups], inner, outer, dtype, pad_rows=5).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_strides_types_and_options(dtype):
    for k, kw in enumerate((dict(pad=8), dict(pad=3), dict(out=F32), dict(otype=torch.int64), dict(bias=False),
                            dict(pad_rows=300), dict(out=F32, pad=1, pad_rows=70, otype=torch.int64))):
        flush_print("grouped", dtype, kw)
        Case([40, 0, 129, 300], 136, 88, dtype, seed=10 * k, **kw).all()
    Case([40, 0, 129], 136, 88, dtype).backward_weight(bias=False)


def test_larger_sides():
    for groups, inner, outer in (([300, 0, 513, 1000], 1024, 512), ([5, 2, 0, 1], 2048, 1040), ([260, 260], 520, 1032)):
        flush_print("grouped", groups, inner, outer)
        Case(groups, inner, outer, BF16, pad_rows=3).all()


@pytest.mark.parametrize("groups,inner,outer,dtype", [
    ([7600, 7400], 2040, 1000, BF16),                          # forward and by input: 256 x 256
    ([1100, 0, 900, 2001], 1016, 1032, F16),                   # 128 x 128
    ([4000 + 13 * e for e in range(16)], 1024, 1000, BF16),    # by weight: 256 x 256
    ([16000], 4088, 1000, BF16),                               # by weight: 256 x 256, rows shared
    ([5000, 9000, 6000], 1001, 515, F16),                      # odd: 256 x 128
    ([700, 20, 0, 3000], 515, 1001, BF16),                     # odd: 64 x 64
])
def test_each_tile(groups, inner, outer, dtype):
    """Sizes at which each tile is the one expected to be fastest, with edges inside it."""
    flush_print("grouped", groups, inner, outer)
    Case(groups, inner, outer, dtype, pad_rows=7).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("groups,inner,outer", [
    ([9000, 4100, 1900], 2041, 1001),      # forward, by input and by weight: 256 x 256, rows shared
    ([2500, 0, 1400, 2100], 1001, 1201),   # forward and by input: 256 x 128
    ([900, 1, 700, 1399], 2047, 901),      # by weight: 128 x 128
    ([300, 0, 7, 393], 515, 77),           # 64 x 64
])
def test_each_tile_at_any_alignment(groups, inner, outer, dtype):
    """As test_each_tile, where rows do not start on 16 bytes or do not end on them."""
    flush_print("grouped", groups, inner, outer)
    Case(groups, inner, outer, dtype, pad_rows=7).all()


@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("inner,outer", [(1, 1), (3, 8), (7, 2), (8, 5), (9, 15), (71, 7), (129, 9), (64, 63)])
def test_narrow_sides(inner, outer, pad):
    """Sides around the 8 values of one load, over several steps of 64 rows; the last group ends the buffers."""
    flush_print("grouped", inner, outer, pad)
    Case([65, 130, 0, 257], inner, outer, BF16, pad=pad).all()


def test_many_experts():
    g = torch.Generator().manual_seed(3)
    groups = [int(n) for n in torch.randint(0, 9, (200,), generator=g)]
    Case(groups, 48, 40, BF16, pad_rows=2).all()
    for n in (63, 64, 65):  # around the experts that one wave counts at a time
        Case(groups[:n], 40, 72, BF16, pad_rows=70).all()


def test_long_group():
    """A weight gradient over many rows next to short ones."""
    Case([20000, 7, 0, 300], 96, 64, BF16).backward_weight()
    Case([20000, 7, 0, 300], 96, 64, F16, out=F32).backward_weight()


def test_no_rows():
    c = Case([0, 0], 40, 24, BF16)
    c.forward()
    c.backward_input()
    c.backward_weight()
    only_pad = Case([0, 0, 0], 64, 64, F16, pad_rows=90)
    only_pad.all()


def test_special_values_stay_in_their_rows():
    """An infinity or a NaN in a row reaches that row's results (and its expert's weights' gradient) only."""
    for inner, outer in ((128, 64), (33, 17)):
        c = Case([40, 70, 20], inner, outer, BF16)
        c.x[45, 3] = float("nan")
        c.x[128, inner - 1] = float("inf")
        y = torch.empty(c.rows, outer, dtype=BF16, device="cuda")
        tbe.tbe_grouped_linear_forward(c.x, c.w, c.b, c.off, y)
        assert (~y.isfinite()).any(1).nonzero()[:, 0].tolist() == [45, 128]
        gw = torch.empty(3, outer, inner, dtype=BF16, device="cuda")
        ws = tbe.workspace(tbe.tbe_grouped_linear_backward_weight_workspace_bytes(c.rows, 3, inner, outer))
        tbe.tbe_grouped_linear_backward_weight(c.x, c.gy, c.off, gw, None, ws)
        assert gw[0].isfinite().all()
        assert (~gw[1].isfinite()).nonzero()[:, 1].unique().tolist() == [3]
        assert (~gw[2].isfinite()).nonzero()[:, 1].unique().tolist() == [inner - 1]


def test_gradients_against_differences():
    c = Case([30, 0, 21], 56, 40, F16, out=F32)
    gx, (gw, gb) = c.backward_input(), c.backward_weight()
    dx, dw, db = draw(c.x.shape, F32, 5).double(), draw(c.w.shape, F32, 6).double(), draw(c.b.shape, F32, 7).double()

    def loss(h):
        total = 0.0
        for e, s in c.spans():
            y = (c.x[s].double() + h * dx[s]) @ (c.w[e].double() + h * dw[e]).t() + c.b[e].double() + h * db[e]
            total = total + (c.gy[s].double() * y).sum()
        return total

    h = 1e-4
    change = (loss(h) - loss(-h)) / (2 * h)  # the loss is of second order: no error but rounding
    terms = [gx.double() * dx, gw.double() * dw, gb.double() * db]
    size = float(sum(t.abs().sum() for t in terms))
    assert abs(float(change - sum(t.sum() for t in terms))) <= (2 * U * (56 / 8 + 32) + 1e-9) * size


def test_repeats_and_graph_replays():
    c = Case([500, 0, 77, 900], 264, 136, BF16, pad_rows=9)
    ws = tbe.workspace(tbe.tbe_grouped_linear_backward_weight_workspace_bytes(c.rows, 4, 264, 136))
    y, gx = torch.empty(c.rows, 136, dtype=BF16, device="cuda"), torch.empty(c.rows, 264, dtype=BF16, device="cuda")
    gw, gb = torch.empty(4, 136, 264, device="cuda"), torch.empty(4, 136, device="cuda")

    def step():
        tbe.tbe_grouped_linear_forward(c.x, c.w, c.b, c.off, y)
        tbe.tbe_grouped_linear_backward_input(c.gy, c.w, c.off, gx)
        tbe.tbe_grouped_linear_backward_weight(c.x, c.gy, c.off, gw, gb, ws)

    outs = (y, gx, gw, gb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    eager = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    scratch = torch.randn(1 << 20, device="cuda")
    for k in range(3):
        for t in outs:
            t.zero_()
        g.replay()
        scratch.mul_(1.5).add_(float(k))
        torch.cuda.synchronize()
        for t, e in zip(outs, eager):
            assert torch.equal(t, e)
