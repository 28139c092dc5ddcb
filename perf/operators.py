"""The dense tower's operators over the pooled embeddings, as cases that can be measured.

Three operators of include/tbe_tower.h, each in the form in which a training or serving program calls it:
  norm     layer norm of rows (the pooled embeddings of a bag, or one table's slice of them): forward, and backward
           with the gradients of the scale and the shift
  expert   a linear layer for each expert on rows that are grouped by expert: forward, and backward with the
           gradients of the input, the weights and the biases
  adamw    one AdamW step over all the tower's tensors, with states of 32 bits or of 8 bits

With own = False run() computes them from elementary torch operations in 32 bits; with own = True it calls the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 128             # values of an 8-bit state that share one scale
BETA1, BETA2, ADAM_EPS, LR = 0.9, 0.999, 1e-8, 1e-3
NORM_EPS = 1e-5


# ----------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one request's pooled rows at serving time: latency alone
        {"name": "norm forward, one request", "op": "norm_forward", "rows": 32, "width": 1024, "x": "f32", "y": "bf16"},
        # all pooled rows of a training batch: 32 tables of width 128 for 131072 bags, normalised into the tower's type
        {"name": "norm forward, pooled rows", "op": "norm_forward", "rows": 131072, "width": 4096, "x": "f32", "y": "bf16"},
        # the same rows' gradient: the pooled output's gradient is fp32, as the embedding backward takes it
        {"name": "norm backward, pooled rows", "op": "norm_backward", "rows": 131072, "width": 4096, "x": "f32", "y": "bf16"},
        # a layer inside the tower whose width is odd: rows start at any alignment
        {"name": "norm backward, odd width", "op": "norm_backward", "rows": 10007, "width": 1001, "x": "bf16", "y": "bf16"},
        # a few requests, each for its own market's expert: the weights' bytes decide
        {"name": "expert forward, few rows", "op": "expert_forward", "rows": 24, "pad": 8, "experts": 8, "inner": 1024,
         "outer": 512, "skew": 0.5, "empty": 2, "type": "bf16"},
        # a training batch over 16 experts of unequal popularity
        {"name": "expert forward, training batch", "op": "expert_forward", "rows": 131072, "pad": 0, "experts": 16,
         "inner": 4096, "outer": 1024, "skew": 0.6, "empty": 0, "type": "bf16"},
        # its backward: the gradients of the rows, the weights and the biases
        {"name": "expert backward, training batch", "op": "expert_backward", "rows": 131072, "pad": 0, "experts": 16,
         "inner": 4096, "outer": 1024, "skew": 0.6, "empty": 0, "type": "bf16", "grad": "bf16"},
        # odd sizes, experts that no row chose, weight gradients kept in fp32
        {"name": "expert backward, odd sizes", "op": "expert_backward", "rows": 5003, "pad": 21, "experts": 13, "inner": 1000,
         "outer": 515, "skew": 1.0, "empty": 3, "type": "f16", "grad": "f32"},
        # a small tower's step: 24 tensors, launch-bound
        {"name": "adamw, small tower", "op": "adamw", "count": 24, "total": 300_000, "p": "f32", "g": "f32", "state": 32,
         "master": False},
        # a large tower in fp32
        {"name": "adamw, large tower", "op": "adamw", "count": 120, "total": 200_000_000, "p": "f32", "g": "f32", "state": 32,
         "master": False},
        # a bf16 tower with fp32 master weights
        {"name": "adamw, master weights", "op": "adamw", "count": 61, "total": 50_000_000, "p": "bf16", "g": "bf16",
         "state": 32, "master": True},
        # a large bf16 tower whose states are held in 8 bits
        {"name": "adamw, states of 8 bits", "op": "adamw", "count": 120, "total": 200_000_000, "p": "bf16", "g": "bf16",
         "state": 8, "master": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a power of two, a multiple of 40, or any number."""
    kind = rng.randrange(3)
    if kind == 0:
        return 1 << rng.randint(max(0, math.ceil(math.log2(lo))), math.floor(math.log2(hi)))
    n = _log(rng, lo, hi)
    return max(40, n // 40 * 40) if kind == 1 else n | 1


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "expert_forward", "expert_backward", "adamw"])
    if op.startswith("norm"):
        width = _width(rng, 4, 16384)
        rows = _log(rng, 16, max(32, min(1 << 21, (1 << 28) // width)))
        return {"op": op, "rows": rows, "width": width, "x": rng.choice(["f32", "f16", "bf16"]),
                "y": rng.choice(["f32", "f16", "bf16"])}
    if op.startswith("expert"):
        inner, outer, experts = _width(rng, 24, 4096), _width(rng, 1, 2048), rng.choice([1, 4, 8, 13, 16, 32])
        rows = _log(rng, 8, 65536)
        case = {"op": op, "rows": rows, "pad": rng.choice([0, 0, rng.randrange(200)]), "experts": experts, "inner": inner,
                "outer": outer, "skew": round(rng.uniform(0.0, 1.2), 2), "empty": rng.randrange(1 + experts // 3),
                "type": rng.choice(["f16", "bf16"])}
        if op == "expert_backward":
            case["grad"] = rng.choice(["f32", case["type"]])
        return case
    p, master = rng.choice([("f32", False), ("bf16", False), ("bf16", True), ("f16", True)])
    return {"op": op, "count": rng.randint(3, 150), "total": _log(rng, 100_000, 150_000_000), "p": p,
            "g": rng.choice([p, "f32"]), "state": rng.choice([32, 8]), "master": master}


def _sizes(case):
    """The tensors' sizes, from the case alone: half of them vectors, the others share the rest."""
    r = np.random.RandomState(case["count"] * 7919 + case["total"] % 10007)
    few = case["count"] // 2
    small = r.randint(1, max(2, min(4096, case["total"] // (2 * case["count"]))), few)
    share = r.dirichlet(np.full(case["count"] - few, 2.0)) * max(0, case["total"] - int(small.sum()))
    return [int(n) for n in r.permutation(np.concatenate([small, np.maximum(1, share.astype(np.int64))]))]


def _groups(case, seed):
    """Rows of each expert, from the seed: some experts have none, the others get a share by popularity."""
    r = np.random.RandomState(seed % (1 << 31))
    n = case["experts"]
    share = 1.0 / np.arange(1, n + 1) ** case["skew"]
    share[n - case["empty"]:] = 0.0
    return [int(c) for c in r.multinomial(case["rows"], r.permutation(share / share.sum()))]


def work(case):
    if case["op"].startswith("norm"):
        n, x, y = case["rows"] * case["width"], DTYPE[case["x"]].itemsize, DTYPE[case["y"]].itemsize
        if case["op"] == "norm_forward":
            return {"bytes": n * (x + y) + 8 * case["rows"] + 8 * case["width"], "flops": 8 * n}
        return {"bytes": n * (2 * x + y) + 8 * case["rows"] + 12 * case["width"], "flops": 16 * n}
    if case["op"].startswith("expert"):
        m, k, n, e = case["rows"], case["inner"], case["outer"], DTYPE[case["type"]].itemsize
        padded, used = m + case["pad"], min(m, case["experts"])
        if case["op"] == "expert_forward":
            return {"bytes": e * (m * k + used * (k * n + n) + padded * n), "flops": 2 * m * k * n}
        g = DTYPE[case["grad"]].itemsize
        return {"bytes": e * (m * (k + n) + used * k * n + padded * k) + g * case["experts"] * (k + 1) * n,
                "flops": 4 * m * k * n}
    total, p, g = sum(_sizes(case)), DTYPE[case["p"]].itemsize, DTYPE[case["g"]].itemsize
    each = 2 * p + g + (16 if case["state"] == 32 else 4 + 4) + ((8 - p) if case["master"] else 0)
    return {"bytes": total * each + (total // 32 if case["state"] == 8 else 0), "flops": 16 * total}


# ----------------------------------------------------------------------------------------------------------------
# what a program has in hand before the call
# ----------------------------------------------------------------------------------------------------------------
def _normal(shape, seed, dtype, scale=1.0, shift=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).mul_(scale).add_(shift).to(dtype)


def _flat(sizes, seed, dtype, scale, positive=False):
    """One buffer for all tensors, each at a multiple of BLOCK; what lies between them is zero."""
    at = np.concatenate([[0], np.cumsum([-(-n // BLOCK) * BLOCK for n in sizes])])
    flat = _normal((int(at[-1]),), seed, torch.float32, scale)
    if positive:
        flat.square_()
    for a, b, n in zip(at[:-1], at[1:], sizes):
        flat[int(a) + n:int(b)] = 0
    return flat.to(dtype), [int(a) for a in at[:-1]]


def prepare(case, seed):
    s = {"case": case, "op": case["op"]}
    if case["op"].startswith("norm"):
        rows, width, tx, ty = case["rows"], case["width"], DTYPE[case["x"]], DTYPE[case["y"]]
        # pooled embeddings: sums of a few lookups, each row around a value of its own
        s["x"] = (_normal((rows, width), seed, torch.float32, 0.3) + _normal((rows, 1), seed + 1, torch.float32, 0.2)).to(tx)
        s["weight"] = _normal((width,), seed + 2, torch.float32, 0.1, 1.0)
        s["bias"] = _normal((width,), seed + 3, torch.float32, 0.1)
        s["mean"], s["rstd"] = (torch.empty(rows, device=DEV) for _ in range(2))
        if case["op"] == "norm_forward":
            s["y"] = torch.empty(rows, width, dtype=ty, device=DEV)
        else:
            s["grad_y"] = _normal((rows, width), seed + 4, ty, 0.01)
            mean = s["x"].float().mean(1, keepdim=True)
            s["mean"], s["rstd"] = mean[:, 0], ((s["x"].float() - mean).square().mean(1) + NORM_EPS).rsqrt()
            s["grad_x"] = torch.empty(rows, width, dtype=tx, device=DEV)
            s["grad_weight"], s["grad_bias"] = (torch.empty(width, device=DEV) for _ in range(2))
            s["workspace"] = _workspace("tbe_layer_norm_backward_workspace_bytes", rows, width)
    elif case["op"].startswith("expert"):
        n, k, experts, t = case["outer"], case["inner"], case["experts"], DTYPE[case["type"]]
        s["groups"] = _groups(case, seed)
        s["rows"], s["padded"] = case["rows"], case["rows"] + case["pad"]
        s["offsets"] = torch.tensor([0] + list(np.cumsum(s["groups"])), dtype=torch.int32, device=DEV)
        s["x"] = _normal((s["padded"], k), seed, t)
        s["weight"] = _normal((experts, n, k), seed + 1, t, k ** -0.5)
        if case["op"] == "expert_forward":
            s["bias"] = _normal((experts, n), seed + 2, t, 0.1)
            s["y"] = torch.empty(s["padded"], n, dtype=t, device=DEV)
        else:
            s["grad_y"] = _normal((s["padded"], n), seed + 3, t, 0.01)
            s["grad_x"] = torch.empty(s["padded"], k, dtype=t, device=DEV)
            s["grad_weight"] = torch.empty(experts, n, k, dtype=DTYPE[case["grad"]], device=DEV)
            s["grad_bias"] = torch.empty(experts, n, dtype=DTYPE[case["grad"]], device=DEV)
            s["workspace"] = _workspace("tbe_grouped_linear_backward_weight_workspace_bytes", s["padded"], experts, k, n)
    else:
        sizes = _sizes(case)
        master, at = _flat(sizes, seed, torch.float32, 0.05)
        s["param"] = master.to(DTYPE[case["p"]])
        s["master"] = master if case["master"] else None
        s["grad"], _ = _flat(sizes, seed + 1, DTYPE[case["g"]], 1e-2)
        m, _ = _flat(sizes, seed + 2, torch.float32, 3e-3)
        v, _ = _flat(sizes, seed + 3, torch.float32, 1e-2, positive=True)
        # vectors (scales, shifts, biases) are not decayed
        decay = [0.01 if n > 4096 else 0.0 for n in sizes]
        s["decay"] = torch.tensor(np.repeat(decay, [-(-n // BLOCK) for n in sizes]), dtype=torch.float32, device=DEV)
        s["step"] = 100
        if case["state"] == 32:
            s["m"], s["v"], s["m_scale"], s["v_scale"] = m, v, None, None
        else:
            (s["m"], s["m_scale"]), (s["v"], s["v_scale"]) = _pack_m(m), _pack_v(v)
            s["m_out"], s["v_out"] = (torch.zeros(m.numel(), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        s["plan"] = _adamw_plan(s, sizes, at, decay)
    return s


def _workspace(name, *sizes):
    """The library's workspace; on a tree that has no such entry point there is none."""
    if not own:
        return None
    import bwd_tbe_fwd_amd as tbe
    return tbe.workspace(getattr(tbe, name)(*sizes))


def _adamw_plan(s, sizes, at, decay):
    if not own:
        return None
    import bwd_tbe_fwd_amd as tbe

    def views(flat, unit=1):
        return None if flat is None else [flat[a // unit:a // unit + -(-n // unit)] for a, n in zip(at, sizes)]

    s["m_views"], s["v_views"] = views(s.get("m_out")), views(s.get("v_out"))
    return tbe.AdamWTensors(views(s["param"]), views(s["grad"]), views(s["m"]), views(s["v"]), weight_decay=decay,
                            masters=views(s["master"]), exp_avg_scales=views(s["m_scale"], BLOCK),
                            exp_avg_sq_scales=views(s["v_scale"], BLOCK))


# ----------------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import bwd_tbe_fwd_amd as tbe
    op = s["op"]
    if op == "norm_forward":
        tbe.tbe_layer_norm_forward(s["x"], s["weight"], s["bias"], NORM_EPS, s["y"], s["mean"], s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_backward":
        tbe.tbe_layer_norm_backward(s["x"], s["grad_y"], s["mean"], s["rstd"], s["weight"], s["grad_x"], s["grad_weight"],
                                    s["grad_bias"], s["workspace"])
        return {"grad_x": s["grad_x"], "grad_weight": s["grad_weight"], "grad_bias": s["grad_bias"]}
    if op == "expert_forward":
        tbe.tbe_grouped_linear_forward(s["x"], s["weight"], s["bias"], s["offsets"], s["y"])
        return {"y": s["y"]}
    if op == "expert_backward":
        tbe.tbe_grouped_linear_backward_input(s["grad_y"], s["weight"], s["offsets"], s["grad_x"])
        tbe.tbe_grouped_linear_backward_weight(s["x"], s["grad_y"], s["offsets"], s["grad_weight"], s["grad_bias"],
                                               s["workspace"])
        return {"grad_x": s["grad_x"], "grad_weight": s["grad_weight"], "grad_bias": s["grad_bias"]}
    s["step"] += 1
    tbe.tbe_adamw_step(s["plan"], s["step"], LR, BETA1, BETA2, ADAM_EPS)
    out = {"param": s["param"], "exp_avg": s["m"], "exp_avg_sq": s["v"], "master": s["master"]}
    if s["m_scale"] is not None:
        tbe.tbe_adamw_state_read(s["plan"], s["m_views"], s["v_views"])
        out.update(exp_avg=s["m_out"], exp_avg_sq=s["v_out"])
    return out


def _run_plain(s):
    op = s["op"]
    if op == "norm_forward":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        x = x - mean
        rstd = (x.square().mean(1, keepdim=True) + NORM_EPS).rsqrt()
        return {"y": (x * rstd * s["weight"] + s["bias"]).to(s["y"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "norm_backward":
        rstd, g = s["rstd"][:, None], s["grad_y"].float()
        hat = (s["x"].float() - s["mean"][:, None]) * rstd
        d = g * s["weight"]
        d = (d - d.mean(1, keepdim=True) - hat * (d * hat).mean(1, keepdim=True)) * rstd
        return {"grad_x": d.to(s["x"].dtype), "grad_weight": (g * hat).sum(0), "grad_bias": g.sum(0)}
    if op == "expert_forward":
        x, w, b = s["x"][:s["rows"]].float(), s["weight"].float(), s["bias"].float()
        y = torch.cat([xe @ we.t() + be for xe, we, be in zip(x.split(s["groups"]), w, b)])
        return {"y": torch.cat([y, y.new_zeros(s["padded"] - s["rows"], y.shape[1])]).to(s["y"].dtype)}
    if op == "expert_backward":
        x, g, w = s["x"][:s["rows"]].float(), s["grad_y"][:s["rows"]].float(), s["weight"].float()
        xs, gs = x.split(s["groups"]), g.split(s["groups"])
        gx = torch.cat([ge @ we for ge, we in zip(gs, w)])
        gw, gb = torch.stack([ge.t() @ xe for xe, ge in zip(xs, gs)]), torch.stack([ge.sum(0) for ge in gs])
        t = s["grad_weight"].dtype
        return {"grad_x": torch.cat([gx, gx.new_zeros(s["padded"] - s["rows"], gx.shape[1])]).to(s["x"].dtype),
                "grad_weight": gw.to(t), "grad_bias": gb.to(t)}
    s["step"] += 1
    eight = s["m_scale"] is not None
    m, v = (_open_m(s["m"], s["m_scale"]), _open_v(s["v"], s["v_scale"])) if eight else (s["m"], s["v"])
    g = s["grad"].float()
    # products and sums each rounded by themselves, so that the 8-bit codes are the same everywhere
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    size = LR / (1 - BETA1 ** s["step"])
    p = (s["param"] if s["master"] is None else s["master"]).float().view(-1, BLOCK)
    p = (p * (1 - LR * s["decay"])[:, None]).view(-1) - size * m / (v.sqrt() / math.sqrt(1 - BETA2 ** s["step"]) + ADAM_EPS)
    s["param"].copy_(p)
    if s["master"] is not None:
        s["master"].copy_(p)
    if eight:
        for name, (code, scale) in (("m", _pack_m(m)), ("v", _pack_v(v))):
            s[name].copy_(code)
            s[name + "_scale"].copy_(scale)
        m, v = _open_m(s["m"], s["m_scale"]).bfloat16(), _open_v(s["v"], s["v_scale"]).bfloat16()
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return {"param": s["param"], "exp_avg": m, "exp_avg_sq": v, "master": s["master"]}


# States of 8 bits: each BLOCK values share a power of two, 2^(e - 127), e the biased exponent of the largest magnitude
# within [24, 250].  A first moment is held as e4m3 of value * 2^7 / 2^(e - 127); a second moment, never negative, as
# an unsigned number of 5 exponent and 3 mantissa bits of value / 2^(e - 127), and one above zero never becomes zero.
def _scale(blocks):
    e = (blocks.abs().amax(1).view(torch.int32) >> 23).clamp(24, 250)
    return e, ((254 - e) << 23).view(torch.float32)[:, None]


def _pack_m(m):
    e, inverse = _scale(m.view(-1, BLOCK))
    return (m.view(-1, BLOCK) * inverse * 128.0).to(torch.float8_e4m3fn).view(torch.uint8).view(-1), e.to(torch.uint8)


def _open_m(code, e):
    one = (e.to(torch.int32) << 23).view(torch.float32)[:, None]
    return (code.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * 2.0 ** -7 * one).view(-1)


def _pack_v(v):
    e, inverse = _scale(v.view(-1, BLOCK))
    bits = (v.view(-1, BLOCK) * inverse).view(torch.int32)
    code = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - 776
    return torch.where(bits > 0, code.clamp(1, 254), 0).to(torch.uint8).view(-1), e.to(torch.uint8)


def _open_v(code, e):
    one = (e.to(torch.int32) << 23).view(torch.float32)[:, None]
    value = torch.where(code > 0, (code.to(torch.int32) + 776) << 20, 0).view(torch.float32)
    return (value.view(-1, BLOCK) * one).view(-1)


# ----------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_forward":
        parts = []
        for x in s["x"].split(8192):
            x = x.double()
            var, mean = torch.var_mean(x, 1, correction=0)
            r = 1.0 / torch.sqrt(var + NORM_EPS)
            y = torch.addcmul(s["bias"].double(), (x - mean[:, None]) / torch.sqrt(var + NORM_EPS)[:, None], s["weight"].double())
            parts.append((y, mean, r))
        y, mean, rstd = (torch.cat(p) for p in zip(*parts))
        return {"y": y, "mean": mean, "rstd": rstd}
    if case["op"] == "norm_backward":
        w = s["weight"].double().requires_grad_()
        b = s["bias"].double().requires_grad_()
        grads = []
        for x, g in zip(s["x"].split(8192), s["grad_y"].split(8192)):
            x = x.double().requires_grad_()
            var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
            y = (x - mean) / torch.sqrt(var + NORM_EPS) * w + b
            y.backward(g.double())
            grads.append(x.grad)
        return {"grad_x": torch.cat(grads), "grad_weight": w.grad, "grad_bias": b.grad}
    if case["op"].startswith("expert"):
        x, w, at = s["x"].double(), s["weight"].double(), s["offsets"].tolist()
        if case["op"] == "expert_forward":
            y = x.new_zeros(s["padded"], case["outer"])
            for e in range(case["experts"]):
                rows = slice(at[e], at[e + 1])
                y[rows] = torch.addmm(s["bias"][e].double(), x[rows], w[e].transpose(0, 1))
            return {"y": y}
        g = s["grad_y"].double()
        gx, gw, gb = torch.zeros_like(x), torch.zeros_like(w), w.new_zeros(w.shape[:2])
        for e in range(case["experts"]):
            rows = slice(at[e], at[e + 1])
            gx[rows] = torch.mm(g[rows], w[e])
            gw[e] = torch.mm(x[rows].transpose(0, 1), g[rows]).transpose(0, 1)
            gb[e] = torch.ones(1, at[e + 1] - at[e], dtype=torch.float64, device=DEV).mm(g[rows])[0]
        return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    t = s["step"] + 1
    g = s["grad"].double()
    if case["state"] == 8:
        m, v = _open_m(s["m"], s["m_scale"]).double(), _open_v(s["v"], s["v_scale"]).double()
    else:
        m, v = s["m"].double(), s["v"].double()
    m = torch.lerp(m, g, 1 - BETA1)
    v = torch.lerp(v, g.square(), 1 - BETA2)
    p = (s["param"] if s["master"] is None else s["master"]).double()
    decay = s["decay"].double().repeat_interleave(BLOCK)
    p = p - LR * decay * p - LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + ADAM_EPS)
    out = {"param": p, "exp_avg": m, "exp_avg_sq": v, "master": p if case["master"] else None}
    if case["state"] == 8:
        out.update(exp_avg=_round_m(m), exp_avg_sq=_round_v(v))
    return out


def _unit(blocks):
    """The power of two of each block's largest magnitude, as a column."""
    top = blocks.abs().amax(1, keepdim=True)
    return torch.exp2((torch.frexp(top)[1] - 1).clamp(-103, 123).double())


def _four_bits(x, lowest):
    """x rounded to four significant bits, ties to even, with no step below 2^(lowest - 3)."""
    step = torch.exp2((torch.frexp(x)[1] - 1).clamp(min=lowest).double() - 3)
    return torch.round(x / step) * step


def _round_m(m):
    blocks = m.view(-1, BLOCK)
    unit = _unit(blocks) / 128
    return (_four_bits(blocks / unit, -6) * unit).view(-1)


def _round_v(v):
    blocks = v.view(-1, BLOCK)
    unit = _unit(blocks)
    least = 1.125 * 2.0 ** -30
    rounded = _four_bits(blocks / unit, -1000).clamp(min=least)
    return (torch.where(blocks > 0, rounded, 0.0) * unit).view(-1)
