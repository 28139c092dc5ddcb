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


def test_workspace_of_the_largest_batch_serves_smaller_ones():
    rng = random.Random(2)
    for rows, experts, inner, outer in [(1 << 20, 1, 4096, 1024), (1 << 18, 8, 256, 128), (100000, 16, 1024, 1024), *shapes(200, 3)]:
        steps = sorted({rng.randint(0, rows) for _ in range(200)} | set(range(0, rows + 1, 64)) if rows < 20000 else
                       {rng.randint(0, rows) for _ in range(600)})
        sizes = [need(r, experts, inner, outer) for r in steps] + [need(rows, experts, inner, outer)]
        assert sizes == sorted(sizes), (rows, experts, inner, outer)
    assert need(511, 4, 1024, 1024) == 0
    # the sizes at which a smaller batch once needed more
    assert need(4032, 1, 4096, 1024) <= need(4160, 1, 4096, 1024)
    assert need(163776, 1, 4096, 1024) <= need(196544, 1, 4096, 1024)
