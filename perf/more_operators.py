"""Workloads for what surrounds an expert block's products: the routing of tokens with its
balance loss and per-expert counts, the rows moved to the experts and back, and the gated
activation with its 8-bit checkpoint -- forward and backward.

A case is a dict of plain values.  ``prepare`` makes what a caller has in hand, ``run`` is one
pass -- in plain fp32 torch operations, or through the library where ``own`` is set -- ``exact``
the same result from the formulas in fp64, and ``work`` the bytes and operations that the pass
cannot do without.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 32  # values that share a scale in an 8-bit checkpoint


def listed():
    return [
        # decoding: 8 sequences, each token to 2 of 8 experts
        dict(name="route_token", op="route", type="bf16", tokens=8, experts=8, k=2, score="softmax",
             normalize=True, scale=1.0, masked=0.0, balance=0.0, align=1),
        # a training batch over 64 experts, 3 % of it padding, with the balance loss
        dict(name="route_64e", op="route", type="f32", tokens=16384, experts=64, k=8, score="softmax",
             normalize=True, scale=1.0, masked=0.03, balance=0.01, align=1),
        # a large batch over 256 experts scored one by one, groups padded for the quantized products
        dict(name="route_256e", op="route", type="f32", tokens=65536, experts=256, k=8,
             score="sigmoid", normalize=True, scale=2.5, masked=0.0, balance=1e-4, align=128),
        # the router's gradient, weights not normalised; an odd number of tokens
        dict(name="route_backward_64e", op="route_backward", type="bf16", tokens=16381, experts=64,
             k=8, score="softmax", normalize=False, scale=1.0, masked=0.03, balance=0.01),
        # and that of the large batch
        dict(name="route_backward_256e", op="route_backward", type="f32", tokens=65536, experts=256,
             k=8, score="sigmoid", normalize=True, scale=2.5, masked=0.0, balance=1e-4),
        # decoding: 8 tokens' rows to 2 experts each
        dict(name="dispatch_token", op="dispatch", type="bf16", tokens=8, cols=4096, experts=8, k=2,
             masked=0.0, align=1),
        # a training batch to 8 experts, groups padded with zero rows for the quantized products
        dict(name="dispatch_8e", op="dispatch", type="bf16", tokens=8192, cols=4096, experts=8, k=2,
             masked=0.0, align=128),
        # the weighted sums of 8 experts' rows each
        dict(name="combine_64e", op="combine", type="f16", tokens=4096, cols=2048, experts=64, k=8,
             masked=0.0),
        # and the gradients of such sums, of the rows and of the weights
        dict(name="combine_backward_8e", op="combine_backward", type="bf16", tokens=8192, cols=4096,
             experts=8, k=2, masked=0.02, align=1),
        # decoding: the activation alone, nothing kept for a backward pass
        dict(name="act_token", op="act", type="bf16", rows=16, cols=14336, act="silu", gated=True,
             keep=False),
        # the activation of a training batch, its inputs kept in 8 bits
        dict(name="act_8e", op="act", type="bf16", rows=16384, cols=14336, act="silu", gated=True,
             keep=True),
        # its backward pass from such a checkpoint over 64 small experts; the activation itself is
        # made again for the weight gradient
        dict(name="act_backward_64e", op="act_backward", type="f16", rows=32768, cols=1408,
             act="gelu", gated=True, again=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = [max(work(case)[m] for case in listed()) for m in ("bytes", "flops")]
    op = rng.choice(["route", "route_backward", "dispatch", "combine", "combine_backward", "act",
                     "act_backward"])
    while True:
        case = _draw(rng, op)
        cost = work(case)
        if cost["bytes"] <= most[0] and cost["flops"] <= most[1]:
            return case


def _draw(rng, op):
    if op.startswith("route"):
        experts = rng.choice([_log(rng, 2, 256), 8, 64, 128, 256])
        case = dict(op=op, type=rng.choice(["bf16", "f16", "f32"]), tokens=_log(rng, 1, 65536),
                    experts=experts, k=rng.randint(1, min(8, experts)),
                    score=rng.choice(["softmax", "sigmoid"]), normalize=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.0, 0.05]),
                    balance=rng.choice([0.0, 1e-3, 0.01]))
        if op == "route":
            case["align"] = rng.choice([1, 1, 128])
        return case
    if op.startswith("act"):
        rows, cols = _log(rng, 1, 32768), 8 * _log(rng, 8, 2048)
        if rng.random() < 0.15:  # now and then of any width
            cols -= rng.randint(1, 7)
        case = dict(op=op, type=rng.choice(["bf16", "f16"]), rows=rows, cols=cols,
                    act=rng.choice(["silu", "gelu"]), gated=rng.random() < 0.8)
        case["keep" if op == "act" else "again"] = rng.random() < 0.7
        return case
    tokens, cols = _log(rng, 1, 16384), 8 * _log(rng, 8, 1024)
    if rng.random() < 0.15:
        cols -= rng.randint(1, 7)
    case = dict(op=op, type=rng.choice(["bf16", "f16", "f32"]), tokens=tokens, cols=cols,
                experts=rng.choice([8, 16, 64, 128]), k=rng.randint(1, 8),
                masked=rng.choice([0.0, 0.0, 0.05]))
    if op != "combine":
        case["align"] = rng.choice([1, 1, 128])
    return case


# ------------------------------------------------------------------ sizes
def _blocks(case):
    return (case["cols"] + BLOCK - 1) // BLOCK


def _rows_capacity(case):
    """Rows that a batch can need: each token's k, and every group's padding."""
    return case["tokens"] * case["k"] + case["experts"] * (case["align"] - 1)


def _live(case):
    """Tokens that are no padding, and the rows that they take among the experts."""
    tokens = case["tokens"] - int(case["masked"] * case["tokens"])
    return tokens, tokens * case["k"]


def work(case):
    op = case["op"]
    e = SIZE[case["type"]]
    if op.startswith("route"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        mask = T if case["masked"] else 0
        if op == "route":  # logits -> experts, weights, rows; counts and offsets, slopes
            return {"bytes": T * E * e + mask + 12 * T * k + 28 * E, "flops": (k + 6) * T * E}
        # logits, experts, the weights' gradients -> the logits'
        return {"bytes": 2 * T * E * e + 8 * T * k + 4 * E, "flops": 10 * T * E}
    if op.startswith("act"):
        n, parts = case["rows"] * case["cols"], 2 if case["gated"] else 1
        kept = parts * (n + case["rows"] * _blocks(case))  # values and scales
        if op == "act":
            return {"bytes": (parts + 1) * n * e + (kept if case["keep"] else 0), "flops": 12 * n}
        return {"bytes": kept + (1 + parts + (1 if case["again"] else 0)) * n * e, "flops": 20 * n}
    T, k, H = case["tokens"], case["k"], case["cols"]
    tokens, rows = _live(case)
    if op == "dispatch":  # (the padding rows depend on the sizes: half a step a group)
        pad = case["experts"] * (case["align"] - 1) // 2
        return {"bytes": (tokens + rows + pad) * H * e + 4 * T * k, "flops": 0}
    if op == "combine":
        return {"bytes": (T + rows) * H * e + 8 * T * k, "flops": 2 * rows * H}
    pad = case["experts"] * (case["align"] - 1) // 2
    return {"bytes": (tokens + 2 * rows + pad) * H * e + 12 * T * k, "flops": 3 * rows * H}


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, scale=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _logits(case, gen):
    """A router's logits: some experts are liked better than others."""
    E = case["experts"]
    x = _normal(gen, (case["tokens"], E), 1.5) + _normal(gen, (E,), 0.5)
    return x.to(TYPES[case["type"]])


def _mask(case, gen):
    """1 for a token, 0 for padding; none where the whole batch counts."""
    if not case["masked"]:
        return None
    mask = torch.ones(case["tokens"], dtype=torch.uint8, device="cuda")
    order = torch.randperm(case["tokens"], generator=gen, device="cuda")
    mask[order[:int(case["masked"] * case["tokens"])]] = 0
    return mask


def _chosen(logits, k, mask):
    """The k experts of each token by logit, the lower one first where two are alike."""
    E = logits.shape[1]
    bits = (logits.float() + 0.0).view(torch.int32)  # -0 is 0
    rank = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)
    key = rank * E + (E - 1 - torch.arange(E, device=logits.device))
    expert = (E - 1 - torch.remainder(key.topk(k, dim=1).values, E)).to(torch.int32)
    return expert if mask is None else torch.where(mask[:, None] != 0, expert, -1)


def _row_plan(expert, E, align, capacity, last_dim):
    """Rows sorted by expert, a token's before the next one's: tokens per expert, row of each
    choice, and the groups' sizes and offsets."""
    flat = expert.reshape(-1).to(torch.int64)
    flat = torch.where(flat < 0, E, flat)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    counts.scatter_add_(0, flat, torch.ones_like(flat))
    sizes = (counts[:E] + align - 1) // align * align
    ends = sizes.cumsum(0)
    starts = torch.cat([ends - sizes, ends.new_zeros(1)])  # the last: of choices that are none
    by_expert, order = torch.sort(flat, stable=True)
    before = torch.cat([counts.new_zeros(1), counts.cumsum(0)[:-1]])
    at = torch.arange(flat.numel(), device=flat.device) - before[by_expert] + starts[by_expert]
    at = torch.where((by_expert < E) & (at < capacity), at, -1)
    row_of = torch.empty_like(flat)
    row_of[order] = at
    kept = ends.clamp(max=capacity)
    sizes = kept - torch.cat([kept.new_zeros(1), kept[:-1]])
    ws = torch.cat([sizes, sizes.new_zeros(1), kept * last_dim])
    return counts[:E].to(torch.int32), row_of.reshape(expert.shape).to(torch.int32), ws


def _power(e):
    """2^e for whole numbers from -127 to 127."""
    return torch.where(e > -127, ((e.to(torch.int32) + 127) << 23).view(torch.float32), 2.0 ** -127)


def _quantized(x):
    """[rows, cols] -> E4M3 values and, for each 32 of a row, the exponent byte of their scale:
    the least power of two that brings the largest of them to 448 or less."""
    rows, cols = x.shape
    blocks = (cols + BLOCK - 1) // BLOCK
    v = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    m, e = torch.frexp(v.abs().amax(2))  # m in [0.5, 1), 448 = 0.875 * 2^9
    e = torch.where(m > 0, e - 9 + (m > 0.875).to(e.dtype), -127).clamp(-127, 127)
    q = (v * _power(-e)[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(rows, -1)[:, :cols].contiguous(), (e + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s, op = {"case": dict(case)}, case["op"]
    if op.startswith("route"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        s["logits"], s["mask"] = _logits(case, gen), _mask(case, gen)
        if op == "route":
            new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
            s["expert"], s["row_of"] = new((T, k), torch.int32), new((T, k), torch.int32)
            s["weight"], s["counts"] = new((T, k), torch.float32), new(E, torch.int32)
            s["group_ws"] = new(2 * E + 1, torch.int64)
            s["loss"], s["slope"] = new(1, torch.float32), new(E, torch.float32)
            if own:
                from moe_grouped_block_gb300 import mxg
                s["ws"] = mxg.alloc_route_workspace(T, E, k)
        else:  # what the forward pass kept
            s["expert"] = _chosen(s["logits"], k, s["mask"])
            s["dweight"] = _normal(gen, (T, k), 0.1)
            s["dloss"] = torch.full((1,), 1.0, device="cuda")
            counts, _, _ = _row_plan(s["expert"], E, 1, T * k, 1)
            share = counts.float() / counts.sum()
            s["slope"] = case["balance"] * E * share / max(1, _live(case)[0])
            s["dlogits"] = torch.empty_like(s["logits"])
        return s
    t = TYPES[case["type"]]
    if op.startswith("act"):
        rows, cols, parts = case["rows"], case["cols"], 2 if case["gated"] else 1
        # gate and up as one product leaves them, side by side
        wide = _normal(gen, (rows, parts * cols), 1.2, t)
        if op == "act":
            s["gate"], s["up"] = wide[:, :cols], wide[:, cols:] if case["gated"] else None
            s["h"] = torch.empty((rows, cols), dtype=t, device="cuda")
            if case["keep"]:
                s["q"] = torch.empty((rows, parts * cols), dtype=torch.uint8, device="cuda")
                s["sf"] = torch.empty((rows, parts * _blocks(case)), dtype=torch.uint8, device="cuda")
        else:
            kept = [_quantized(wide[:, i * cols:(i + 1) * cols]) for i in range(parts)]
            s["q"] = torch.cat([q.view(torch.uint8) for q, _ in kept], 1)
            s["sf"] = torch.cat([sf for _, sf in kept], 1)
            s["dh"] = _normal(gen, (rows, cols), 0.02, t)
            s["dwide"] = torch.empty((rows, parts * cols), dtype=t, device="cuda")
            s["h"] = torch.empty((rows, cols), dtype=t, device="cuda") if case["again"] else None
        return s
    # the plan of a batch: who goes where
    route = dict(case, type="f32")
    mask = _mask(case, gen)
    expert = _chosen(_logits(route, gen), case["k"], mask)
    align = case.get("align", 1)
    s["capacity"] = _rows_capacity(dict(case, align=align))
    s["counts"], s["row_of"], s["group_ws"] = _row_plan(expert, case["experts"], align, s["capacity"],
                                                        case["cols"])
    T, H, k = case["tokens"], case["cols"], case["k"]
    if op == "dispatch":
        s["x"] = _normal(gen, (T, H), 1.0, t)
        s["rows"] = torch.zeros((s["capacity"], H), dtype=t, device="cuda")
        return s
    w = torch.rand((T, k), generator=gen, device="cuda") + 0.05
    s["weight"] = w / w.sum(1, keepdim=True)
    s["y_rows"] = _normal(gen, (s["capacity"], H), 0.7, t)
    if op == "combine":
        s["y"] = torch.empty((T, H), dtype=t, device="cuda")
    else:
        s["dy"] = _normal(gen, (T, H), 0.02, t)
        s["dy_rows"] = torch.zeros((s["capacity"], H), dtype=t, device="cuda")
        s["dweight"] = torch.empty((T, k), device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"route": _own_route, "route_backward": _own_route_backward, "dispatch": _own_dispatch,
                "combine": _own_combine, "combine_backward": _own_combine_backward, "act": _own_act,
                "act_backward": _own_act_backward}[op](s)
    return {"route": _plain_route, "route_backward": _plain_route_backward,
            "dispatch": _plain_dispatch, "combine": _plain_combine,
            "combine_backward": _plain_combine_backward, "act": _plain_act,
            "act_backward": _plain_act_backward}[op](s)


def _score(mxg, case):
    return mxg.MXG_SCORE_SOFTMAX if case["score"] == "softmax" else mxg.MXG_SCORE_SIGMOID


def _own_route(s):
    from moe_grouped_block_gb300 import mxg
    c = s["case"]
    mxg.mxg_route(s["logits"], s["expert"], s["weight"], s["counts"], mask=s["mask"],
                  score=_score(mxg, c), normalize=c["normalize"], scale=c["scale"],
                  balance=c["balance"], loss=s["loss"], slope=s["slope"], row_of=s["row_of"],
                  group_ws=s["group_ws"], align=c["align"], rows_capacity=_rows_capacity(c),
                  last_dim=1, workspace=s["ws"])
    return {k: s[k] for k in ("expert", "weight", "counts", "loss", "slope", "row_of", "group_ws")}


def _scores(logits, c):
    """What a router makes of its logits: the scores, and their shares of a token's whole."""
    x = logits.float()
    s = torch.sigmoid(x) if c["score"] == "sigmoid" else (x - x.amax(1, keepdim=True)).exp()
    p = s / s.sum(1, keepdim=True)
    return (s if c["score"] == "sigmoid" else p), p


def _plain_route(s):
    c, E, k = s["case"], s["case"]["experts"], s["case"]["k"]
    score, p = _scores(s["logits"], c)
    expert = _chosen(s["logits"], k, s["mask"])
    weight = score.gather(1, expert.clamp(min=0).to(torch.int64))
    if c["normalize"]:
        weight = weight / weight.sum(1, keepdim=True)
    weight = weight * c["scale"]
    live = p.new_tensor(float(c["tokens"]))
    if s["mask"] is not None:
        taken = s["mask"][:, None] != 0
        weight, p = torch.where(taken, weight, 0.0), torch.where(taken, p, 0.0)
        live = taken.sum().float()
    counts, row_of, ws = _row_plan(expert, E, c["align"], _rows_capacity(c), 1)
    slope = c["balance"] * E * (counts.float() / counts.sum()) / live
    return {"expert": expert, "weight": weight, "counts": counts,
            "loss": (slope * p.sum(0)).sum().reshape(1), "slope": slope, "row_of": row_of,
            "group_ws": ws}


def _own_route_backward(s):
    from moe_grouped_block_gb300 import mxg
    c = s["case"]
    mxg.mxg_route_backward(s["logits"], s["expert"], s["dlogits"], dweight=s["dweight"],
                           score=_score(mxg, c), normalize=c["normalize"], scale=c["scale"],
                           slope=s["slope"], dloss=s["dloss"])
    return s["dlogits"]


def _plain_route_backward(s):
    c = s["case"]
    score, p = _scores(s["logits"], c)
    at = s["expert"].clamp(min=0).to(torch.int64)
    dw = s["dweight"] * c["scale"]
    chosen = score.gather(1, at)
    if c["normalize"]:
        whole = chosen.sum(1, keepdim=True)
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / whole) / whole
    a = (s["slope"] * s["dloss"]).expand_as(p)
    balance = a - (a * p).sum(1, keepdim=True)
    if c["score"] == "softmax":  # p is the score: one product with its derivative for both
        both = a.scatter_add(1, at, dw)
        d = p * (both - (both * p).sum(1, keepdim=True))
    else:
        d = score * (1 - score) * torch.zeros_like(p).scatter_add(1, at, dw)
        d = d + p * (1 - score) * balance
    if s["mask"] is not None:
        d = torch.where(s["mask"][:, None] != 0, d, 0.0)
    return d.to(s["logits"].dtype)


def _own_dispatch(s):
    from moe_grouped_block_gb300 import mxg
    pad = s["case"]["align"] > 1
    mxg.mxg_dispatch(s["x"], s["row_of"], s["rows"], counts=s["counts"] if pad else None,
                     group_ws=s["group_ws"] if pad else None)
    return s["rows"]


def _plain_dispatch(s):
    at = s["row_of"].reshape(-1).to(torch.int64)
    who = torch.arange(at.numel(), device=at.device) // s["case"]["k"]
    rows = torch.zeros((s["capacity"] + 1, s["case"]["cols"]), dtype=s["x"].dtype, device=at.device)
    rows[torch.where(at < 0, s["capacity"], at)] = s["x"][who]
    return rows[:-1]


def _own_combine(s):
    from moe_grouped_block_gb300 import mxg
    mxg.mxg_combine(s["y_rows"], s["row_of"], s["y"], weight=s["weight"])
    return s["y"]


def _plain_combine(s):
    at = s["row_of"].to(torch.int64)
    w = torch.where(at < 0, 0.0, s["weight"])
    rows = s["y_rows"][at.clamp(min=0)].float()
    return (rows * w[:, :, None]).sum(1).to(s["y"].dtype)


def _own_combine_backward(s):
    from moe_grouped_block_gb300 import mxg
    pad = s["case"]["align"] > 1
    mxg.mxg_combine_backward(s["dy"], s["row_of"], s["weight"], s["dy_rows"], y_rows=s["y_rows"],
                             dweight=s["dweight"], counts=s["counts"] if pad else None,
                             group_ws=s["group_ws"] if pad else None)
    return {"dy_rows": s["dy_rows"], "dweight": s["dweight"]}


def _plain_combine_backward(s):
    at = s["row_of"].to(torch.int64)
    none = at < 0
    dy = s["dy"].float()
    rows = s["y_rows"][at.clamp(min=0)].float()
    dweight = torch.where(none, 0.0, (rows * dy[:, None]).sum(2))
    d = torch.zeros((s["capacity"] + 1, dy.shape[1]), dtype=s["dy"].dtype, device=dy.device)
    each = (dy[:, None] * s["weight"][:, :, None]).to(s["dy"].dtype)
    d[torch.where(none, s["capacity"], at).reshape(-1)] = each.reshape(-1, dy.shape[1])
    d = d[:-1].contiguous()
    return {"dy_rows": d, "dweight": dweight}


def _act(mxg, case):
    return mxg.MXG_ACT_SILU if case["act"] == "silu" else mxg.MXG_ACT_GELU_TANH


def _own_act(s):
    from moe_grouped_block_gb300 import mxg
    keep = s["case"]["keep"]
    mxg.mxg_gated_act(s["gate"], s["h"], up=s["up"], act=_act(mxg, s["case"]),
                      q=s["q"] if keep else None, sf=s["sf"] if keep else None)
    if not keep:
        return {"h": s["h"]}
    return {"h": s["h"], "q": s["q"].view(torch.float8_e4m3fn), "sf": s["sf"]}


# gelu(g) = g sigmoid(z(g)) with the tanh form's z, silu the same with z = g
GELU_A, GELU_B = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


def _sigmoid_and_slope(g, act):
    """sigmoid(z(g)) and z'(g)."""
    if act == "silu":
        return torch.sigmoid(g), 1.0
    return torch.sigmoid(GELU_A * (g + GELU_B * g * g * g)), GELU_A * (1 + 3 * GELU_B * g * g)


def _plain_act(s):
    c = s["case"]
    g = s["gate"].float()
    h = g * _sigmoid_and_slope(g, c["act"])[0]
    if c["gated"]:
        h = h * s["up"].float()
    got = {"h": h.to(s["h"].dtype)}
    if c["keep"]:
        kept = [_quantized(s["gate"])] + ([_quantized(s["up"])] if c["gated"] else [])
        got["q"] = torch.cat([q.view(torch.uint8) for q, _ in kept], 1).view(torch.float8_e4m3fn)
        got["sf"] = torch.cat([sf for _, sf in kept], 1)
    return got


def _own_act_backward(s):
    from moe_grouped_block_gb300 import mxg
    c = s["case"]
    F, d = c["cols"], s["dwide"]
    mxg.mxg_gated_act_backward(s["q"], s["sf"], s["dh"], d[:, :F], dup=d[:, F:] if c["gated"] else None,
                               act=_act(mxg, c), h=s["h"])
    return {"dwide": d, "h": s["h"]} if c["again"] else {"dwide": d}


def _restored(q, sf, cols):
    """The values that a checkpoint stands for."""
    scale = _power(sf.to(torch.int32) - 127)
    return q.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(BLOCK, 1)[:, :cols]


def _plain_act_backward(s):
    c = s["case"]
    F, B = c["cols"], _blocks(c)
    dh = s["dh"].float()
    g = _restored(s["q"][:, :F], s["sf"][:, :B], F)
    sig, dz = _sigmoid_and_slope(g, c["act"])
    a, da = g * sig, sig + g * sig * (1 - sig) * dz
    if c["gated"]:
        u = _restored(s["q"][:, F:], s["sf"][:, B:], F)
        d, h = torch.cat([dh * u * da, dh * a], 1), a * u
    else:
        d, h = dh * da, a
    got = {"dwide": d.to(s["dh"].dtype)}
    if c["again"]:
        got["h"] = h.to(s["dh"].dtype)
    return got


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    return {"route": _exact_route, "route_backward": _exact_route_backward,
            "dispatch": _exact_dispatch, "combine": _exact_combine,
            "combine_backward": _exact_combine_backward, "act": _exact_act,
            "act_backward": _exact_act_backward}[op](s)


def _exact_shares(x, c):
    """(scores, shares) of fp64 logits, from their logarithms."""
    if c["score"] == "softmax":
        p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
        return p, p
    s = torch.exp(torch.nn.functional.logsigmoid(x))
    return s, s / s.sum(1, keepdim=True)


def _exact_weight(x, expert, c):
    score, p = _exact_shares(x, c)
    w = torch.stack([score[torch.arange(len(x), device=x.device), e] for e in expert.unbind(1)], 1)
    if c["normalize"]:
        w = w / w.sum(1, keepdim=True)
    return c["scale"] * w, p


def _exact_route(s):
    c, E, k = s["case"], s["case"]["experts"], s["case"]["k"]
    x = s["logits"].double()
    live = torch.ones(len(x), dtype=torch.bool, device=x.device)
    if s["mask"] is not None:
        live = s["mask"].bool()
    expert = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    weight, p = _exact_weight(x, expert, c)
    weight[~live] = 0
    counts = torch.bincount(expert[live].reshape(-1), minlength=E)
    expert[~live] = -1
    slope = c["balance"] * E * counts.double() / (counts.sum() * live.sum())
    # whole numbers from the sizes alone, one choice after the other, per expert
    sizes = [-(-int(n) // c["align"]) * c["align"] for n in counts]
    ends = [sum(sizes[:e + 1]) for e in range(E)]
    row_of = torch.full((expert.numel(),), -1, dtype=torch.int32, device=x.device)
    flat = expert.reshape(-1)
    for e in range(E):
        at = (flat == e).nonzero()[:, 0]
        row_of[at] = torch.arange(len(at), dtype=torch.int32, device=x.device) + ends[e] - sizes[e]
    return {"expert": expert.to(torch.int32), "weight": weight, "counts": counts.to(torch.int32),
            "loss": (slope * p[live].sum(0)).sum().reshape(1), "slope": slope,
            "row_of": row_of.reshape(expert.shape),
            "group_ws": torch.tensor(sizes + [0] + ends, device=x.device)}


def _exact_route_backward(s):
    c = s["case"]
    x = s["logits"].double().requires_grad_()
    live = (s["expert"][:, 0] >= 0).double()
    weight, p = _exact_weight(x, s["expert"].clamp(min=0).to(torch.int64), c)
    rows = (weight * s["dweight"].double()).sum(1) + (p * s["slope"].double()).sum(1) * s["dloss"].double()
    return torch.autograd.grad((rows * live).sum(), x)[0]


def _exact_dispatch(s):
    out = torch.zeros(s["rows"].shape, dtype=torch.float64, device="cuda")
    for at in s["row_of"].unbind(1):
        t = (at >= 0).nonzero()[:, 0]
        out.index_copy_(0, at[t].to(torch.int64), s["x"][t].double())
    return out


def _exact_combine(s):
    out = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    for j, at in enumerate(s["row_of"].unbind(1)):
        t = (at >= 0).nonzero()[:, 0]
        out[t] += s["y_rows"][at[t].to(torch.int64)].double() * s["weight"][t, j, None].double()
    return out


def _exact_combine_backward(s):
    d = torch.zeros(s["dy_rows"].shape, dtype=torch.float64, device="cuda")
    dweight = torch.zeros(s["weight"].shape, dtype=torch.float64, device="cuda")
    for j, at in enumerate(s["row_of"].unbind(1)):
        t = (at >= 0).nonzero()[:, 0]
        dy, at = s["dy"][t].double(), at[t].to(torch.int64)
        d[at] = dy * s["weight"][t, j, None].double()
        dweight[t, j] = torch.einsum("th,th->t", dy, s["y_rows"][at].double())
    return {"dy_rows": d, "dweight": dweight}


def _exact_activation(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g.pow(3))))


def _exact_kept(x):
    """E4M3 values by rounding to a grid of 4 bits a binade (half to even), and exponent bytes."""
    qs, bytes_ = [], []
    for part in x.split(BLOCK, 1):
        v = part.double()
        top = v.abs().amax(1, keepdim=True)
        e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)), -127).clamp(-127, 127)
        v = v * torch.exp2(-e)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        qs.append(torch.round(v / step) * step)
        bytes_.append((e + 127).to(torch.uint8))
    return torch.cat(qs, 1), torch.cat(bytes_, 1)


def _exact_act(s):
    c = s["case"]
    h = _exact_activation(s["gate"].double(), c["act"])
    if c["gated"]:
        h = h * s["up"].double()
    if not c["keep"]:
        return {"h": h}
    kept = [_exact_kept(s["gate"])] + ([_exact_kept(s["up"])] if c["gated"] else [])
    return {"h": h, "q": torch.cat([q for q, _ in kept], 1), "sf": torch.cat([b for _, b in kept], 1)}


def _exact_values(q, sf):
    """Bytes of sign, 4 bits of exponent and 3 of fraction, times a power of two for each 32."""
    b = q.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
    v = torch.where(b > 127, -v, v)
    scale = torch.exp2(sf.double() - 127)
    return torch.cat([part * scale[:, i:i + 1] for i, part in enumerate(v.split(BLOCK, 1))], 1)


def _exact_act_backward(s):
    c = s["case"]
    F, B = c["cols"], _blocks(c)
    leaves = [_exact_values(s["q"][:, :F], s["sf"][:, :B]).requires_grad_()]
    h = _exact_activation(leaves[0], c["act"])
    if c["gated"]:
        leaves.append(_exact_values(s["q"][:, F:], s["sf"][:, B:]).requires_grad_())
        h = h * leaves[1]
    d = torch.cat(torch.autograd.grad(h, leaves, s["dh"].double()), 1)
    return {"dwide": d, "h": h.detach()} if c["again"] else {"dwide": d}
