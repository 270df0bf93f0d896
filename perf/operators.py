"""Workloads for the 16-bit operators of an expert block: the grouped products, the norms
around the block with its gate and residual, and the clipping of the gradients.

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
EPS = 1e-6
CLIP_EPS = 1e-6


def listed():
    return [
        # the smallest grouped call: a block of toy size, where a call's latency is all there is
        dict(name="tiny_fprop", op="gemm", mode="fprop", type="bf16", out="f32", G=4, K=256, N=256,
             rows=512, live=3, layout=0),
        # decoding: 8 tokens, 2 experts each, through the up projection of an 8-expert layer
        dict(name="token_fprop_8e", op="gemm", mode="fprop", type="bf16", out="bf16", G=8, K=4096,
             N=14336, rows=16, live=7, layout=1),
        # decoding with 64 small experts: 12 tokens, 8 experts each
        dict(name="token_fprop_64e", op="gemm", mode="fprop", type="f16", out="f16", G=64, K=2048,
             N=1408, rows=96, live=49, layout=2),
        # a training or prefill batch through the 8-expert layer
        dict(name="fprop_8e", op="gemm", mode="fprop", type="bf16", out="bf16", G=8, K=4096, N=14336,
             rows=16384, live=8, layout=3),
        # the activation gradient of the 64-expert layer, one expert without tokens
        dict(name="dgrad_64e", op="gemm", mode="dgrad", type="f16", out="f16", G=64, K=2048, N=1408,
             rows=32768, live=63, layout=4),
        # the weight gradient of the 8-expert layer into fp32; group sizes of any value
        dict(name="wgrad_8e", op="gemm", mode="wgrad", type="bf16", out="f32", G=8, K=4096, N=14336,
             rows=16381, live=8, layout=5),
        # the norms around one block when a single token is decoded
        dict(name="norm_token", op="norm", way="forward", type="bf16", res="bf16", rows=1, cols=4096,
             gate="none", scale=1.0),
        # the same for a training batch, with a gate per channel
        dict(name="norm_forward", op="norm", way="forward", type="bf16", res="bf16", rows=16384,
             cols=4096, gate="col", scale=1.0),
        # and its backward pass, with the gradients of both weights and of the gate
        dict(name="norm_backward", op="norm", way="backward", type="bf16", res="bf16", rows=16384,
             cols=4096, gate="col", scale=1.0),
        # an fp32 residual stream with the router's weight as the gate of a row; an odd row count
        dict(name="norm_backward_f32", op="norm", way="backward", type="bf16", res="f32", rows=2777,
             cols=7168, gate="row", scale=0.5),
        # clipping the gradients of one small layer: norms, biases and projections of odd sizes
        dict(name="clip_layer", op="clip", type="bf16", to="f32", tensors=48, least=1, most=262147,
             layout=6, ratio=0.37),
        # clipping the expert gradients of one 8-expert layer (three projections an expert)
        dict(name="clip_8e", op="clip", type="bf16", to="bf16", tensors=24, least=14336 * 4096,
             most=14336 * 4096, layout=7, ratio=0.37),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        case = _draw(rng)
        if 3072 not in case.values():
            return case


def _draw(rng):
    op = rng.choice(["gemm", "gemm", "norm", "clip"])
    layout = rng.randrange(1 << 20)
    if op == "gemm":
        mode = rng.choice(["fprop", "dgrad", "wgrad"])
        kind = rng.choice(["bf16", "f16"])
        G = _log(rng, 1, 64)
        while True:  # row strides are multiples of 8 elements (16 bytes)
            N, K, rows = 8 * _log(rng, 8, 1792), 8 * _log(rng, 8, 896), _log(rng, 1, 32768)
            if G * N * K <= 8 * 4096 * 14336 and rows * N * K <= 16384 * 4096 * 14336:
                break
        return dict(op=op, mode=mode, type=kind, out=rng.choice([kind, "f32"]), G=G, K=K, N=N,
                    rows=rows, live=rng.randint(1, min(G, rows)), layout=layout)
    if op == "norm":
        kind = rng.choice(["bf16", "f16"])
        while True:
            rows, cols = _log(rng, 1, 32768), _log(rng, 64, 16384)
            cols -= cols % 8 if rng.random() < 0.75 else 0  # one in four of any width
            if rows * cols <= 16384 * 4096:
                break
        return dict(op=op, way=rng.choice(["forward", "backward"]), type=kind,
                    res=rng.choice([kind, "f32"]), rows=rows, cols=cols,
                    gate=rng.choice(["none", "row", "col", "full"]),
                    scale=round(rng.uniform(0.1, 1.0), 3))
    tensors = _log(rng, 1, 400)
    most = _log(rng, 64, 1 << 24)
    return dict(op=op, type=rng.choice(["bf16", "f16", "f32"]), to=rng.choice(["same", "f32"]),
                tensors=tensors, least=max(1, most // rng.choice([1, 16, 1024])), most=most,
                layout=layout, ratio=rng.choice([0.013, 0.37, 2.0]))


# ------------------------------------------------------------------ sizes
def _group_sizes(case):
    """Rows per expert: `live` experts share the rows unevenly, each with at least one."""
    rng = random.Random(case["layout"])
    sizes = [0] * case["G"]
    who = rng.sample(range(case["G"]), case["live"])
    weight = [rng.expovariate(1.0) + 0.05 for _ in who]
    spare, left = case["rows"] - len(who), case["rows"]
    for g, w in zip(who, weight):
        sizes[g] = 1 + int(spare * w / sum(weight))
        left -= sizes[g]
    sizes[who[0]] += left
    return sizes


def _tensor_sizes(case):
    rng = random.Random(case["layout"])
    return [_log(rng, case["least"], case["most"]) for _ in range(case["tensors"])]


def _clip_type(case):
    return case["type"] if case["to"] == "same" else case["to"]


def work(case):
    if case["op"] == "gemm":
        M, N, K, e = case["rows"], case["N"], case["K"], SIZE[case["type"]]
        o = SIZE[case["out"]]
        if case["mode"] == "fprop":
            b = (M * K + case["live"] * N * K) * e + M * N * o
        elif case["mode"] == "dgrad":
            b = (M * N + case["live"] * N * K) * e + M * K * o
        else:
            b = (M * N + M * K) * e + case["G"] * N * K * o
        return {"bytes": b, "flops": 2 * M * N * K}
    if case["op"] == "norm":
        r, c, e, x = case["rows"], case["cols"], SIZE[case["type"]], SIZE[case["res"]]
        gate = {"none": 0, "row": 4 * r, "col": e * c, "full": e * r * c}[case["gate"]]
        if case["way"] == "forward":  # x, y -> x', n
            return {"bytes": r * c * (2 * x + 2 * e) + 2 * c * e + gate, "flops": 10 * r * c}
        dgate = {"none": 0, "row": 4 * r, "col": 4 * c, "full": e * r * c}[case["gate"]]
        # x', y, dx', dn -> dx, dy and the weights' gradients
        return {"bytes": r * c * (3 * x + 3 * e) + 2 * c * (e + 4) + gate + dgate,
                "flops": 24 * r * c}
    n = sum(_tensor_sizes(case))
    return {"bytes": n * (SIZE[case["type"]] + SIZE[_clip_type(case)]), "flops": 3 * n}


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, scale=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": dict(case)}
    if case["op"] == "gemm":
        t, M, N, K, G = TYPES[case["type"]], case["rows"], case["N"], case["K"], case["G"]
        sizes = _group_sizes(case)
        s["sizes"] = sizes
        if case["mode"] != "dgrad":
            s["x"] = _normal(gen, (M, K), 1.0, t)
        if case["mode"] != "fprop":
            s["dy"] = _normal(gen, (M, N), 1e-3 if case["type"] == "bf16" else 0.05, t)
        if case["mode"] != "wgrad":
            s["w"] = _normal(gen, (G, N, K), 0.02, t)
        shape = {"fprop": (M, N), "dgrad": (M, K), "wgrad": (G, N, K)}[case["mode"]]
        s["c"] = torch.empty(shape, dtype=TYPES[case["out"]], device="cuda")
        # rows per expert as the router leaves them on the device, in the library's workspace
        # layout: G sizes, then the G + 1 row offsets
        offsets = [0]
        for m in sizes:
            offsets.append(offsets[-1] + m)
        s["group_ws"] = torch.tensor(sizes + offsets, dtype=torch.int64, device="cuda")
    elif case["op"] == "norm":
        t, x, r, c = TYPES[case["type"]], TYPES[case["res"]], case["rows"], case["cols"]
        s["x"] = _normal(gen, (r, c), 2.0, x)
        s["y"] = _normal(gen, (r, c), 0.7, t)
        s["w_post"] = (1.0 + _normal(gen, (c,), 0.1)).to(t)
        s["w_pre"] = (1.0 + _normal(gen, (c,), 0.1)).to(t)
        s["gate"] = {"none": lambda: None,
                     "row": lambda: torch.rand((r,), generator=gen, device="cuda"),
                     "col": lambda: _normal(gen, (c,), 0.5, t),
                     "full": lambda: torch.rand((r, c), generator=gen, device="cuda").to(t)}[case["gate"]]()
        if case["way"] == "forward":
            s["x_out"], s["n"] = torch.empty_like(s["x"]), torch.empty_like(s["y"])
        else:
            s["dx_out"], s["dn"] = _normal(gen, (r, c), 0.02, x), _normal(gen, (r, c), 0.02, t)
            s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.empty_like(s["y"])
            s["dw_post"] = torch.empty(c, device="cuda")
            s["dw_pre"] = torch.empty(c, device="cuda")
            s["dgate"] = {"none": None, "row": torch.empty(r, device="cuda"),
                          "col": torch.empty(c, device="cuda"),
                          "full": torch.empty_like(s["y"])}[case["gate"]]
            if own:
                from moe_grouped_block_gb300 import mxg
                s["ws"] = mxg.alloc_block_norm_workspace(r, c)
    else:
        t, to = TYPES[case["type"]], TYPES[_clip_type(case)]
        sizes = _tensor_sizes(case)
        rng = random.Random(case["layout"] + 1)
        # gradients of different layers differ by orders of magnitude
        s["grads"] = [_normal(gen, (n,), 10.0 ** rng.uniform(-4, -2), t) for n in sizes]
        # every result starts on a 16-byte boundary of one buffer, as an optimizer keeps them
        starts, total = [], 0
        for n in sizes:
            starts.append(total)
            total += (n + 7) // 8 * 8
        s["flat"] = torch.zeros(total, dtype=to, device="cuda")
        s["out"] = [s["flat"][a:a + n] for a, n in zip(starts, sizes)]
        s["norm"] = torch.empty(1, device="cuda")
        expected = math.sqrt(sum(float(g[:1 << 16].float().square().mean()) * g.numel()
                                 for g in s["grads"]))
        s["max_norm"] = case["ratio"] * expected
        if own:
            from moe_grouped_block_gb300 import mxg
            s["list"] = mxg.grad_list(s["grads"], s["out"])
            s["ws"] = mxg.alloc_grad_workspace()
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"gemm": _own_gemm, "norm": _own_norm, "clip": _own_clip}[op](s)
    return {"gemm": _plain_gemm, "norm": _plain_norm, "clip": _plain_clip}[op](s)


def _own_gemm(s):
    from moe_grouped_block_gb300 import mxg
    c = s["case"]
    mode = {"fprop": mxg.MXG_FPROP_TN, "dgrad": mxg.MXG_DGRAD_NN, "wgrad": mxg.MXG_WGRAD_NT}[c["mode"]]
    a = s["x"] if c["mode"] == "fprop" else s["dy"]
    b = s["x"] if c["mode"] == "wgrad" else s["w"]
    mxg.mxg_grouped_gemm_16bit(mode, a, b, s["group_ws"], c["G"], c["rows"], c["N"], c["K"], C=s["c"])
    return s["c"]


def _plain_gemm(s):
    c, sizes = s["case"], s["sizes"]
    if c["mode"] == "wgrad":
        dy, x = s["dy"].float().split(sizes), s["x"].float().split(sizes)
        return torch.stack([(a.t() @ b).to(s["c"].dtype) for a, b in zip(dy, x)])
    if c["mode"] == "fprop":
        return torch.cat([(a @ w.float().t()).to(s["c"].dtype)
                          for a, w in zip(s["x"].float().split(sizes), s["w"]) if len(a)])
    return torch.cat([(a @ w.float()).to(s["c"].dtype)
                      for a, w in zip(s["dy"].float().split(sizes), s["w"]) if len(a)])


def _own_norm(s):
    from moe_grouped_block_gb300 import mxg
    c = s["case"]
    mode = {"none": mxg.MXG_GATE_NONE, "row": mxg.MXG_GATE_ROW, "col": mxg.MXG_GATE_COL,
            "full": mxg.MXG_GATE_FULL}[c["gate"]]
    if c["way"] == "forward":
        mxg.mxg_block_norm(s["x"], s["y"], w_post=s["w_post"], gate=s["gate"], gate_mode=mode,
                           res_scale=c["scale"], x_out=s["x_out"], w_pre=s["w_pre"], n_out=s["n"],
                           eps=EPS)
        return {"x_out": s["x_out"], "n": s["n"]}
    mxg.mxg_block_norm_backward(s["x"], s["y"], w_post=s["w_post"], gate=s["gate"], gate_mode=mode,
                                res_scale=c["scale"], w_pre=s["w_pre"], eps=EPS,
                                dx_out=s["dx_out"], dn=s["dn"], dx=s["dx"], dy=s["dy"],
                                dw_post=s["dw_post"], dw_pre=s["dw_pre"], dgate=s["dgate"],
                                workspace=s["ws"])
    return {k: s[k] for k in ("dx", "dy", "dw_post", "dw_pre", "dgate") if s[k] is not None}


def _plain_norm(s):
    c = s["case"]
    x, y, gate = s["x"].float(), s["y"].float(), s["gate"]
    w_post, w_pre = s["w_post"].float(), s["w_pre"].float()
    v = torch.full((1, 1), c["scale"], device=x.device)
    if gate is not None:
        v = c["scale"] * (gate.float()[:, None] if c["gate"] == "row" else gate.float())
    yh = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
    if c["way"] == "forward":
        x = x + v * (yh * w_post)
        n = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w_pre
        return {"x_out": x.to(s["x"].dtype), "n": n.to(s["y"].dtype)}
    dn = s["dn"].float()
    rx = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    ry = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
    xh, a = x * rx, dn * w_pre
    t = s["dx_out"].float() + rx * (a - xh * (a * xh).mean(1, keepdim=True))
    b = t * v * w_post
    got = {"dx": t.to(s["x"].dtype),
           "dy": (ry * (b - yh * (b * yh).mean(1, keepdim=True))).to(s["y"].dtype),
           "dw_post": (t * v * yh).sum(0), "dw_pre": (dn * xh).sum(0)}
    dg = c["scale"] * t * yh * w_post
    if c["gate"] == "full":
        got["dgate"] = dg.to(s["y"].dtype)
    elif c["gate"] != "none":
        got["dgate"] = dg.sum(1 if c["gate"] == "row" else 0)
    return got


def _own_clip(s):
    from moe_grouped_block_gb300 import mxg
    mxg.mxg_grad_clip(s["list"], s["max_norm"], s["norm"], s["ws"])
    return {"out": s["flat"], "norm": s["norm"]}


def _plain_clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    factor = torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * factor)
    return {"out": s["flat"], "norm": norm.reshape(1)}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        M, N, K, ends = case["rows"], case["N"], case["K"], [0]
        for m in s["sizes"]:
            ends.append(ends[-1] + m)
        shape = {"fprop": (M, N), "dgrad": (M, K), "wgrad": (case["G"], N, K)}[case["mode"]]
        out = torch.zeros(shape, dtype=torch.float64, device="cuda")
        for g in range(case["G"]):
            rows = slice(ends[g], ends[g + 1])
            if ends[g] == ends[g + 1]:
                continue
            if case["mode"] == "fprop":
                out[rows] = torch.einsum("ik,nk->in", s["x"][rows].double(), s["w"][g].double())
            elif case["mode"] == "dgrad":
                out[rows] = torch.einsum("in,nk->ik", s["dy"][rows].double(), s["w"][g].double())
            else:
                out[g] = torch.einsum("in,ik->nk", s["dy"][rows].double(), s["x"][rows].double())
        return out
    if case["op"] == "norm":
        # the gradients by automatic differentiation of the formulas
        leaf = {k: s[k].double().requires_grad_(case["way"] == "backward")
                for k in ("x", "y", "w_post", "w_pre", "gate") if s[k] is not None}
        unit = lambda z: z / (z.pow(2).mean(-1, keepdim=True) + EPS).sqrt()  # noqa: E731
        add = case["scale"] * unit(leaf["y"]) * leaf["w_post"]
        if case["gate"] != "none":
            add = add * (leaf["gate"].unsqueeze(1) if case["gate"] == "row" else leaf["gate"])
        if case["way"] == "forward":
            x = leaf["x"] + add
            return {"x_out": x, "n": unit(x) * leaf["w_pre"]}
        # x is the block's output here: its own share of the gradient first, then the rest's
        n = unit(leaf["x"]) * leaf["w_pre"]
        dx, dw_pre = torch.autograd.grad(n, (leaf["x"], leaf["w_pre"]), s["dn"].double())
        dx = dx + s["dx_out"].double()
        names = [k for k in ("y", "w_post", "gate") if k in leaf]
        rest = torch.autograd.grad(add, [leaf[k] for k in names], dx)
        return {"dx": dx, "dw_pre": dw_pre,
                **{{"y": "dy", "w_post": "dw_post", "gate": "dgate"}[k]: v for k, v in zip(names, rest)}}
    total = math.fsum(float(torch.dot(g.double(), g.double())) for g in s["grads"])
    norm = math.sqrt(total)
    flat = torch.zeros(s["flat"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for g in s["grads"]:
        flat[start:start + g.numel()] = g.double() * min(1.0, s["max_norm"] / (norm + CLIP_EPS))
        start += (g.numel() + 7) // 8 * 8
    return {"out": flat, "norm": torch.tensor([norm], dtype=torch.float64)}
