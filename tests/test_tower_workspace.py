"""The workspace of the grouped weight gradient: how large it is.  No GPU needed."""
import math
import random

import bwd_tbe_fwd_amd as tbe

need = tbe.tbe_grouped_linear_backward_weight_workspace_bytes


def shapes(count, seed):
    rng = random.Random(seed)

    def size(lo, hi):
        return 1 << rng.randint(int(math.log2(lo)), int(math.log2(hi))) if rng.random() < 0.5 else \
            int(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    for _ in range(count):
        yield size(8, 1 << 21), rng.choice([1, 2, 5, 8, 13, 16, 64, 200]), size(1, 8192), size(1, 8192)


def test_workspace_is_bounded():
    """At most 1 GiB, or an eighth of the operands' bytes."""
    for rows, experts, inner, outer in [(824148, 1, 5204, 4045), (1278924, 5, 3409, 3726), *shapes(20000, 1)]:
        n = need(rows, experts, inner, outer)
        assert n <= max(1 << 30, rows * (inner + outer) * 2 // 8), (rows, experts, inner, outer, n)
