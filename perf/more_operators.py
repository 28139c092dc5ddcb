"""The two ends of a model that reads and predicts the rows of one table, as cases that can be measured.

Two operators of include/tbe_items.h, each in the form in which a training or serving program calls it:
  lookup         one scaled row for each id: forward, and backward as a dense gradient of the table, overwritten or
                 added to the one that is there
  cross entropy  the softmax cross entropy of each row over all items: forward, and backward with the gradients of the
                 rows, of the items' weights and of their biases

With own = False run() computes them from elementary torch operations in 32 bits; with own = True it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ITYPE = {32: torch.int32, 64: torch.int64}


# ----------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one request's items at serving time: latency alone
        {"name": "lookup forward: one request", "op": "lookup_forward", "ids": 64, "items": 131072, "width": 1024,
         "table": "bf16", "y": "bf16", "itype": 32, "pad": 0.0, "skew": 1.0},
        # all positions of a training batch from one of the benchmark's tables of 2M rows, into the tower's type
        {"name": "lookup forward: training batch", "op": "lookup_forward", "ids": 1048576, "items": 2000000, "width": 128,
         "table": "f16", "y": "bf16", "itype": 64, "pad": 0.1, "skew": 0.91},
        # an odd width in fp32: rows start at any alignment
        {"name": "lookup forward: odd width", "op": "lookup_forward", "ids": 20011, "items": 50021, "width": 1001,
         "table": "f32", "y": "f32", "itype": 64, "pad": 0.05, "skew": 1.0},
        # the dense gradient of a vocabulary's table: a few ids have a good part of the positions
        {"name": "lookup backward: training batch", "op": "lookup_backward", "ids": 131072, "items": 131072, "width": 1024,
         "table": "bf16", "y": "bf16", "itype": 64, "pad": 0.1, "skew": 1.0, "add": False},
        # tied weights: the positions' gradient on top of the loss's, in the 16 bits in which that one came
        {"name": "lookup backward: tied weights", "op": "lookup_backward", "ids": 1048576, "items": 2000000, "width": 128,
         "table": "f16", "y": "f16", "itype": 64, "pad": 0.1, "skew": 0.91, "add": True},
        # a small batch of odd sizes, gradients kept in fp32
        {"name": "lookup backward: odd sizes", "op": "lookup_backward", "ids": 517, "items": 3001, "width": 515,
         "table": "f32", "y": "bf16", "itype": 32, "pad": 0.0, "skew": 1.0, "add": False},
        # the scores of one request's continuations: the weights' bytes decide
        {"name": "loss forward: one request", "op": "loss_forward", "rows": 8, "items": 131072, "width": 1024, "type": "bf16",
         "bias": False, "itype": 64, "pad": 0.0, "skew": 1.0},
        # a training batch over a vocabulary
        {"name": "loss forward: training batch", "op": "loss_forward", "rows": 8192, "items": 131072, "width": 1024,
         "type": "bf16", "bias": False, "itype": 64, "pad": 0.1, "skew": 1.0},
        # retrieval: two million items of width 128, popularity corrected by a bias
        {"name": "loss forward: items of a table", "op": "loss_forward", "rows": 2048, "items": 2000000, "width": 128,
         "type": "f16", "bias": True, "itype": 64, "pad": 0.0, "skew": 0.91},
        # the training batch's backward: gradients of the rows and of the vocabulary's weights
        {"name": "loss backward: training batch", "op": "loss_backward", "rows": 8192, "items": 131072, "width": 1024,
         "type": "bf16", "bias": False, "itype": 64, "pad": 0.1, "skew": 1.0, "weights": False},
        # retrieval's backward, a weight for each sample
        {"name": "loss backward: items of a table", "op": "loss_backward", "rows": 2048, "items": 500000, "width": 128,
         "type": "f16", "bias": True, "itype": 64, "pad": 0.0, "skew": 0.91, "weights": True},
        # odd sizes: rows that start at any alignment, a bias, many positions without a target
        {"name": "loss backward: odd sizes", "op": "loss_backward", "rows": 517, "items": 10007, "width": 515, "type": "bf16",
         "bias": True, "itype": 32, "pad": 0.4, "skew": 1.0, "weights": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a power of two, a multiple of 40, or any odd number."""
    kind = rng.randrange(3)
    if kind == 0:
        return 1 << rng.randint(math.ceil(math.log2(lo)), math.floor(math.log2(hi)))
    n = _log(rng, lo, hi)
    return max(40, n // 40 * 40) if kind == 1 else n | 1


def draw(rng):
    op = rng.choice(["lookup_forward", "lookup_backward", "loss_forward", "loss_backward"])
    case = {"op": op, "itype": rng.choice([32, 64]), "pad": rng.choice([0.0, round(rng.uniform(0.0, 0.6), 2)]),
            "skew": round(rng.uniform(0.0, 1.3), 2)}
    if op.startswith("lookup"):
        width = _width(rng, 4, 4096)
        case.update(width=width, ids=_log(rng, 1, max(2, min(1 << 20, (1 << 27) // width))),
                    items=_log(rng, 10, max(20, min(2000000, (1 << 28) // width))),
                    table=rng.choice(["f32", "f16", "bf16"]), y=rng.choice(["f32", "f16", "bf16"]))
        if op == "lookup_backward":
            case["add"] = rng.choice([False, True])
        return case
    width, rows = _width(rng, 8, 2048), _log(rng, 1, 16384)
    most = min(1000000, (1 << 30) // rows, 8192 * 131072 * 1024 // (rows * width))
    case.update(width=width, rows=rows, items=_log(rng, 30, most), type=rng.choice(["f16", "bf16"]),
                bias=rng.choice([False, True]))
    if op == "loss_backward":
        case["weights"] = rng.choice([False, True])
    return case


def work(case):
    v, d = case["items"], case["width"]
    i = case["itype"] // 8
    if case["op"].startswith("lookup"):
        # rows that are read or written: padding reads nothing, and an id's row counts once however often it is asked for
        n, t, y = case["ids"], DTYPE[case["table"]].itemsize, DTYPE[case["y"]].itemsize
        valid = n - int(n * case["pad"])
        rows = int(_distinct(valid, v, case["skew"]))
        if case["op"] == "lookup_forward":
            return {"bytes": rows * d * t + n * d * y + n * i, "flops": valid * d}
        return {"bytes": valid * d * y + (2 * rows if case["add"] else v) * d * t + n * i, "flops": valid * d}
    n, e = case["rows"], DTYPE[case["type"]].itemsize
    valid = n - int(n * case["pad"])
    bias = 4 * v if case["bias"] else 0
    if case["op"] == "loss_forward":
        return {"bytes": (valid + v) * d * e + bias + n * (i + 8), "flops": 2 * valid * v * d}
    return {"bytes": (valid + v) * d * e + (n + v) * d * e + 2 * bias + n * (i + 8), "flops": 6 * valid * v * d}


def _distinct(n, items, skew):
    """Expected number of different ids among n drawn as _ids draws them."""
    k = torch.arange(items + 1, dtype=torch.float64)
    p = _cumulative(k, items, skew).diff()
    return float((1.0 - torch.exp(n * torch.log1p(-p.clamp(max=1 - 1e-12)))).sum())


# ----------------------------------------------------------------------------------------------------------------
# what a program has in hand before the call
# ----------------------------------------------------------------------------------------------------------------
def _normal(shape, seed, dtype, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).mul_(scale).to(dtype)


def _cumulative(rank, items, skew):
    """The share of the ids among the `rank` most popular ones, where popularity falls as (10 + rank)^-skew."""
    if abs(skew - 1.0) < 1e-6:
        return torch.log((10.0 + rank) / 10.0) / math.log((10.0 + items) / 10.0)
    q = 1.0 - skew
    return ((10.0 + rank) ** q - 10.0 ** q) / ((10.0 + items) ** q - 10.0 ** q)


def _ids(n, items, skew, pad, dtype, seed):
    """Ids by popularity, the popular ones spread over the table, and -1 at int(n * pad) places."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    if abs(skew - 1.0) < 1e-6:
        rank = 10.0 * ((10.0 + items) / 10.0) ** u - 10.0
    else:
        q = 1.0 - skew
        rank = (10.0 ** q + u * ((10.0 + items) ** q - 10.0 ** q)) ** (1.0 / q) - 10.0
    rank = rank.long().clamp(0, items - 1)
    step = 2 * (items // 3) + 1
    while math.gcd(step, items) != 1:
        step += 1
    ids = (rank * step + seed) % items
    ids[torch.randperm(n, generator=g, device=DEV)[:int(n * pad)]] = -1
    return ids.to(dtype)


def prepare(case, seed):
    s = {"case": case, "op": case["op"]}
    v, d = case["items"], case["width"]
    if case["op"].startswith("lookup"):
        n, tt, ty = case["ids"], DTYPE[case["table"]], DTYPE[case["y"]]
        s["scale"] = math.sqrt(d)
        s["ids"] = _ids(n, v, case["skew"], case["pad"], ITYPE[case["itype"]], seed)
        if case["op"] == "lookup_forward":
            s["table"] = _normal((v, d), seed + 1, tt, d ** -0.5)
            s["y"] = torch.empty(n, d, dtype=ty, device=DEV)
        else:
            s["grad_y"] = _normal((n, d), seed + 1, ty, 0.01)
            s["add"] = case["add"]
            s["grad_table"] = _normal((v, d), seed + 2, tt, 0.1) if case["add"] else torch.empty(v, d, dtype=tt, device=DEV)
            s["workspace"] = _workspace("tbe_lookup_backward_workspace_bytes", n, v, d)
        return s
    n, t = case["rows"], DTYPE[case["type"]]
    s["scale"] = 1.0 if d > 128 else 0.5
    # rows that a norm has left, and items that make logits of a few units
    s["x"] = _normal((n, d), seed, t)
    s["weight"] = _normal((v, d), seed + 1, t, 2.0 * d ** -0.5)
    s["bias"] = _normal((v,), seed + 2, torch.float32) if case["bias"] else None
    s["targets"] = _ids(n, v, case["skew"], case["pad"], ITYPE[case["itype"]], seed + 3)
    s["lse"] = torch.empty(n, device=DEV)
    if case["op"] == "loss_forward":
        s["loss"] = torch.empty(n, device=DEV)
        s["workspace"] = _workspace("tbe_cross_entropy_forward_workspace_bytes", n, v, d)
        return s
    for rows, lse, targets in zip(s["x"].split(1024), s["lse"].split(1024), s["targets"].split(1024)):
        lse.copy_(torch.where(targets >= 0, _logits(s, rows).logsumexp(1), 0.0))
    valid = n - int(n * case["pad"])
    # the mean over the rows that have a target; fp16 gradients under a loss scale
    s["grad_loss"] = torch.full((n,), (4096.0 if case["type"] == "f16" else 1.0) / max(1, valid), device=DEV)
    if case["weights"]:
        g = torch.Generator(device=DEV).manual_seed(seed + 4)
        s["grad_loss"] *= 0.25 + 1.5 * torch.rand(n, generator=g, device=DEV)
    s["grad_x"], s["grad_weight"] = torch.empty_like(s["x"]), torch.empty_like(s["weight"])
    s["grad_bias"] = torch.empty(v, device=DEV) if case["bias"] else None
    s["workspace"] = _workspace("tbe_cross_entropy_backward_workspace_bytes", n, v, d)
    return s


def _workspace(name, *sizes):
    """The library's workspace; on a tree that has no such entry point there is none."""
    if not own:
        return None
    import bwd_tbe_fwd_amd as tbe
    return tbe.workspace(getattr(tbe, name)(*sizes))


# ----------------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import bwd_tbe_fwd_amd as tbe
    op = s["op"]
    if op == "lookup_forward":
        tbe.tbe_lookup_forward(s["table"], s["ids"], s["scale"], s["y"])
        return {"y": s["y"]}
    if op == "lookup_backward":
        tbe.tbe_lookup_backward(s["ids"], s["grad_y"], s["scale"], s["grad_table"], s["workspace"], accumulate=s["add"])
        return {"grad_table": s["grad_table"]}
    if op == "loss_forward":
        tbe.tbe_cross_entropy_forward(s["x"], s["weight"], s["bias"], s["targets"], s["scale"], s["loss"], s["lse"],
                                      s["workspace"])
        return {"loss": s["loss"], "lse": s["lse"]}
    tbe.tbe_cross_entropy_backward(s["x"], s["weight"], s["bias"], s["targets"], s["scale"], s["lse"], s["grad_loss"],
                                   s["grad_x"], s["grad_weight"], s["grad_bias"], s["workspace"])
    return {"grad_x": s["grad_x"], "grad_weight": s["grad_weight"], "grad_bias": s["grad_bias"]}


def _logits(s, rows):
    logits = (rows.float() @ s["weight"].float().t()).mul_(s["scale"])
    return logits if s["bias"] is None else logits.add_(s["bias"])


def _run_plain(s):
    op = s["op"]
    if op == "lookup_forward":
        there = (s["ids"] >= 0) & (s["ids"] < s["table"].shape[0])
        rows = s["table"][torch.where(there, s["ids"], 0).long()].float() * s["scale"]
        return {"y": torch.where(there[:, None], rows, 0.0).to(s["y"].dtype)}
    if op == "lookup_backward":
        there = (s["ids"] >= 0) & (s["ids"] < s["grad_table"].shape[0])
        grad = torch.zeros(s["grad_table"].shape, device=DEV)
        grad.index_add_(0, s["ids"][there].long(), s["grad_y"][there].float() * s["scale"])
        s["grad_table"].copy_(s["grad_table"].float() + grad if s["add"] else grad)
        return {"grad_table": s["grad_table"]}
    there = (s["targets"] >= 0) & (s["targets"] < s["weight"].shape[0])
    target = torch.where(there, s["targets"], 0).long()[:, None]
    logits = _logits(s, s["x"])
    if op == "loss_forward":
        score = logits.gather(1, target)[:, 0]
        top = logits.max(1, keepdim=True)[0]
        lse = logits.sub_(top).exp_().sum(1).log() + top[:, 0]
        return {"loss": torch.where(there, lse - score, 0.0), "lse": torch.where(there, lse, 0.0)}
    z = logits.sub_(s["lse"][:, None]).exp_()
    z.scatter_add_(1, target, -torch.ones_like(target, dtype=torch.float32))
    z *= torch.where(there, s["grad_loss"], 0.0)[:, None]
    t = s["x"].dtype
    return {"grad_x": (z @ s["weight"].float()).mul_(s["scale"]).to(t),
            "grad_weight": (z.t() @ s["x"].float()).mul_(s["scale"]).to(t),
            "grad_bias": None if s["bias"] is None else z.sum(0)}


# ----------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lookup_forward":
        # a row of zeros behind the table for the ids that name none
        ids = s["ids"].long()
        table = torch.cat([s["table"], s["table"].new_zeros(1, case["width"])])
        return {"y": torch.index_select(table, 0, ids.remainder(case["items"] + 1)).double().mul_(s["scale"])}
    if case["op"] == "lookup_backward":
        # positions by id; every id's sum is a difference of running sums, taken over a few columns at a time
        order = torch.argsort(s["ids"], stable=True)
        ids = s["ids"][order].long()
        order, ids = order[ids >= 0], ids[ids >= 0]
        ends = torch.searchsorted(ids, torch.arange(case["items"] + 1, device=DEV))
        out = torch.empty(case["items"], case["width"], dtype=torch.float64, device=DEV)
        for at in range(0, case["width"], 128):
            columns = slice(at, at + 128)
            grad = s["grad_y"][order, columns].double()
            sums = torch.cat([grad.new_zeros(1, grad.shape[1]), grad.cumsum(0)])
            out[:, columns] = sums[ends].diff(dim=0)
        out *= s["scale"]
        return {"grad_table": out + s["grad_table"].double() if case["add"] else out}
    x, w, t = s["x"].double(), s["weight"].double(), s["targets"].long()
    b = torch.zeros(case["items"], dtype=torch.float64, device=DEV) if s["bias"] is None else s["bias"].double()
    named = torch.logical_and(t >= 0, t < case["items"])
    part = max(1, (1 << 28) // case["items"])
    if case["op"] == "loss_forward":
        loss, lse = [], []
        for rows, ids, has in zip(x.split(part), t.split(part), named.split(part)):
            all_log = torch.log_softmax(torch.addmm(b, rows, w.transpose(0, 1), alpha=s["scale"]), 1)
            picked = all_log[torch.arange(len(ids), device=DEV), ids.clamp(0, case["items"] - 1)]
            loss.append(torch.where(has, -picked, torch.zeros_like(picked)))
            # log p_0 = l_0 - lse
            lse.append(((rows @ w[0]) * s["scale"] + b[0] - all_log[:, 0]) * has)
        return {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    gx, gw, gb = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b)
    for at in range(0, case["rows"], part):
        rows = torch.arange(at, min(at + part, case["rows"]), device=DEV)[named[at:at + part]]
        if len(rows) == 0:
            continue
        p = torch.softmax(torch.addmm(b, x[rows], w.transpose(0, 1), alpha=s["scale"]), 1)
        p[torch.arange(len(rows), device=DEV), t[rows]] -= 1.0
        p *= s["grad_loss"][rows].double()[:, None]
        gx[rows] = torch.mm(p, w) * s["scale"]
        gw.addmm_(p.transpose(0, 1), x[rows], alpha=s["scale"])
        gb += p.sum(0)
    return {"grad_x": gx, "grad_weight": gw, "grad_bias": None if s["bias"] is None else gb}
