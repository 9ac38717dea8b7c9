"""The operators of the MoE block around and inside the layer, as measured cases.

Four operators of include/moe_block.h, each in its plain form (elementary
torch operations) and as the calls a user makes:

  residual_norm           out = a x + b gate * norm(y), h = norm(out): the post-norm of a
                          block's output, its gate and scale, the residual, and the next
                          block's pre-norm
  residual_norm_backward  the gradients of all of its inputs
  grad_clip               the global L2 norm of a layer's gradients, and their clipped copies
  gemm_i8                 activations quantised per token, then the grouped 8-bit integer
                          product with scales for each token and each output channel
                          (optionally with the SwiGLU gate of the up projection)

`own` selects the framework's kernels; otherwise `run` computes the plain form.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
ALIGN = 128  # dispatched segments start on multiples of this many rows


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of the DeepSeek-V3-shaped layer: latency only
        {"name": "norm-decode-n1-d7168", "op": "residual_norm", "n": 1, "d": 7168,
         "dtype": "bf16", "gate_tokens": 0, "stats": False},
        # a training batch of the same layer; each sequence brings its own gate row
        {"name": "norm-n8192-d7168-gate-per-sequence", "op": "residual_norm", "n": 8192,
         "d": 7168, "dtype": "bf16", "gate_tokens": 1024, "stats": True},
        # a small fp32 model with a ragged batch, a gate row for each token
        {"name": "norm-bwd-n777-d192-f32", "op": "residual_norm_backward", "n": 777, "d": 192,
         "dtype": "f32", "gate_tokens": 1},
        # the training step of the dropless top-8-of-64 layer, one learned gate row
        {"name": "norm-bwd-n16384-d2048", "op": "residual_norm_backward", "n": 16384,
         "d": 2048, "dtype": "bf16", "gate_tokens": 0},
        # gradients of the small fp32 expert-choice layer: one tensor per weight
        {"name": "clip-layer-f32-e8-d128-h512", "op": "grad_clip", "layout": "layer", "E": 8,
         "d": 128, "h": 512, "dtype": "f32", "swiglu": False, "max_norm": 1.0},
        # the dropless layer's gradients: large aligned bf16 tensors and the fp32 router's
        {"name": "clip-layer-bf16-e64-d2048-h1024", "op": "grad_clip", "layout": "layer",
         "E": 64, "d": 2048, "h": 1024, "dtype": "bf16", "swiglu": True, "max_norm": 1.0},
        # every expert's matrices as tensors of their own in one flat buffer, at
        # whatever offset they fall (sizes are odd)
        {"name": "clip-flat-bf16-e256-d193-h129", "op": "grad_clip", "layout": "flat",
         "E": 256, "d": 193, "h": 129, "dtype": "bf16", "swiglu": True, "max_norm": 0.5},
        # one token through one expert's down projection
        {"name": "i8-down-n1-k2048-o7168", "op": "gemm_i8", "rows": 1, "E": 1, "k": 2048,
         "n_out": 7168, "act": "none", "dtype": "bf16", "skew": 0.0},
        # decoding 64 tokens, top-8 of 32: the active experts' weights are streamed
        {"name": "i8-up-64x8of32-k7168-swiglu2048", "op": "gemm_i8", "rows": 512, "E": 32,
         "k": 7168, "n_out": 2048, "act": "swiglu", "dtype": "bf16", "skew": 0.7},
        # a short ragged prompt on the small layer: some experts get no token
        {"name": "i8-up-300x8of64-k256-swiglu128", "op": "gemm_i8", "rows": 2400, "E": 64,
         "k": 256, "n_out": 128, "act": "swiglu", "dtype": "bf16", "skew": 1.5},
        # a prompt batch through the dropless layer's down projection
        {"name": "i8-down-16384x8of64-k1024-o2048", "op": "gemm_i8", "rows": 131072, "E": 64,
         "k": 1024, "n_out": 2048, "act": "none", "dtype": "bf16", "skew": 0.1},
        # a prompt batch through the top-2-of-8 layer's up projection
        {"name": "i8-up-8192x2of8-k4096-swiglu14336", "op": "gemm_i8", "rows": 10240, "E": 8,
         "k": 4096, "n_out": 14336, "act": "swiglu", "dtype": "bf16", "skew": 0.05},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(max(round(v / step) * step, lo), hi))


def draw(rng):
    op = rng.choice(["residual_norm", "residual_norm_backward", "grad_clip", "gemm_i8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("residual_norm", "residual_norm_backward"):
        d = _log(rng, 64, 8192) if rng.random() < 0.3 else _log(rng, 64, 8192, 64)
        n = _log(rng, 1, min(16384, (1 << 25) // d))
        case = {"op": op, "n": n, "d": d, "dtype": dtype,
                "gate_tokens": rng.choice([0, 1, _log(rng, 2, 2048)])}
        if op == "residual_norm":
            case["stats"] = rng.random() < 0.5
        return case
    if op == "grad_clip":
        layout = rng.choice(["layer", "flat"])
        E = _log(rng, 1, 200)
        d = _log(rng, 32, 1024) if layout == "flat" else _log(rng, 64, 1024, 64)
        h = _log(rng, 16, 600) if layout == "flat" else _log(rng, 64, 600, 64)
        return {"op": op, "layout": layout, "E": E, "d": d, "h": h, "dtype": dtype,
                "swiglu": rng.random() < 0.5, "max_norm": rng.choice([0.1, 1.0, 1e6])}
    E = _log(rng, 1, 128)
    k = _log(rng, 64, 8192, 16)
    n_out = _log(rng, 64, 8192, 16)
    while E * k * n_out > 1 << 28:
        E = max(E // 2, 1)
    rows = _log(rng, 1, 20000)
    return {"op": op, "rows": rows, "E": E, "k": k, "n_out": n_out,
            "act": rng.choice(["none", "swiglu"]), "dtype": dtype,
            "skew": rng.choice([0.0, 0.3, 1.0])}


# --------------------------------------------------------------------------- inputs
def _dt(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _gate_rows(case):
    t = case["gate_tokens"]
    return 1 if t == 0 else -(-case["n"] // t)


def _prepare_norm(case, seed):
    g, dt, n, d = _gen(seed), _dt(case), case["n"], case["d"]
    s = {"x": (_randn(g, n, d) * 2).to(dt), "y": _randn(g, n, d).to(dt),
         "w_post": 1 + 0.1 * _randn(g, d), "w_next": 1 + 0.1 * _randn(g, d),
         "gate": (0.3 * _randn(g, _gate_rows(case), d)).to(dt)}
    f32 = dict(dtype=torch.float32, device="cuda")
    if case["op"] == "residual_norm":
        s["out"], s["h"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["rstd_post"] = torch.empty(n, **f32) if case["stats"] else None
        s["rstd_next"] = torch.empty(n, **f32) if case["stats"] else None
        return s
    s["dout"], s["dh"] = _randn(g, n, d).to(dt), _randn(g, n, d).to(dt)
    # what the forward left behind: its output (x here) and both inverse norms
    s["rstd_post"] = (s["y"].double().square().mean(1) + EPS).rsqrt().float()
    s["rstd_next"] = (s["x"].double().square().mean(1) + EPS).rsqrt().float()
    s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    s["dgate"] = torch.empty_like(s["gate"])
    s["dw_post"], s["dw_next"] = torch.empty(d, **f32), torch.empty(d, **f32)
    return s


def _shapes(case):
    """(shape, is_router) of each gradient tensor."""
    E, d, h = case["E"], case["d"], case["h"]
    if case["layout"] == "layer":
        up = [(E, h, d)] * (2 if case["swiglu"] else 1)
        return [((d, E), True)] + [(s, False) for s in up] + [((E, d, h), False)]
    up = [(h, d)] * (2 if case["swiglu"] else 1)
    return [(s, False) for s in (up + [(d, h)]) * E]


def _prepare_clip(case, seed):
    g, dt = _gen(seed), _dt(case)
    shapes = _shapes(case)
    if case["layout"] == "layer":
        grads = [(0.01 * _randn(g, *s)).to(torch.float32 if r else dt) for s, r in shapes]
        return {"grads": grads, "clipped": [torch.empty_like(t) for t in grads]}
    sizes = [math.prod(s) for s, _ in shapes]
    flat = (0.01 * _randn(g, sum(sizes))).to(dt)
    to = torch.empty_like(flat)
    return {"grads": [t.view(s) for t, (s, _) in zip(flat.split(sizes), shapes)],
            "clipped": [t.view(s) for t, (s, _) in zip(to.split(sizes), shapes)], "flat": to}


def _segments(case, seed):
    """Rows of each expert (a skewed random share of the batch), the aligned
    first row of each one's segment, and the rows of the buffers: as many as
    the segments can take for any shares."""
    rng = np.random.RandomState(seed % (1 << 31))
    p = np.exp(case["skew"] * rng.standard_normal(case["E"]))
    counts = rng.multinomial(case["rows"], p / p.sum())
    starts = np.concatenate([[0], np.cumsum(-(-counts // ALIGN) * ALIGN)])
    rows = (case["rows"] + case["E"] * (ALIGN - 1)) // ALIGN * ALIGN
    return counts, starts, rows


def _prepare_i8(case, seed):
    g, dt = _gen(seed), _dt(case)
    E, k, o = case["E"], case["k"], case["n_out"]
    counts, starts, rows = _segments(case, seed)
    most = int(counts.max())
    # dispatched rows: real ones, and whatever lies between and behind the segments
    s = {"x": _randn(g, rows, k).to(dt), "rows": rows, "most": most,
         "starts": torch.from_numpy(starts[:-1].astype(np.int32)).cuda(),
         "counts": torch.from_numpy(counts.astype(np.int32)).cuda()}
    for name in ["w1", "w3"][:2 if case["act"] == "swiglu" else 1]:
        s[name] = torch.randint(-127, 128, (E, o, k), generator=g, device="cuda",
                                dtype=torch.int8)
        s[name + "_scale"] = (0.5 + torch.rand((E, o), generator=g, device="cuda")) * (
            1 / (73.0 * math.sqrt(k)))
    s["q"] = torch.empty((rows, k), dtype=torch.int8, device="cuda")
    s["q_scale"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    s["out"] = torch.zeros((rows, o), dtype=dt, device="cuda")
    return s


def prepare(case, seed):
    if case["op"] == "grad_clip":
        s = _prepare_clip(case, seed)
    elif case["op"] == "gemm_i8":
        s = _prepare_i8(case, seed)
    else:
        s = _prepare_norm(case, seed)
    s["case"] = dict(case)
    return s


# --------------------------------------------------------------------------- plain forms
def _rms(v):
    return torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _gate_of(case, gate):
    """The gate of each token: [n, d], or one row for all."""
    t = case["gate_tokens"]
    return gate if t == 0 else gate.repeat_interleave(t, 0)[:case["n"]]


def _plain_norm(case, s):
    x, y = s["x"].float(), s["y"].float()
    r_post = _rms(y)
    out = x + _gate_of(case, s["gate"].float()) * (y * r_post * s["w_post"])
    r_next = _rms(out)
    h = out * r_next * s["w_next"]
    dt = s["x"].dtype
    return {"out": out.to(dt), "h": h.to(dt),
            "rstd_post": r_post[:, 0] if case["stats"] else None,
            "rstd_next": r_next[:, 0] if case["stats"] else None}


def _plain_norm_backward(case, s):
    out, y, dh = s["x"].float(), s["y"].float(), s["dh"].float()
    r_post, r_next = s["rstd_post"][:, None], s["rstd_next"][:, None]
    u = out * r_next
    dn = dh * s["w_next"]
    dx = s["dout"].float() + r_next * (dn - u * (dn * u).mean(1, keepdim=True))
    v = y * r_post
    gate = _gate_of(case, s["gate"].float())
    per_token = dx * v * s["w_post"]
    t = case["gate_tokens"]
    rows = _gate_rows(case)
    pad = torch.nn.functional.pad(per_token, (0, 0, 0, rows * max(t, 1) - case["n"] if t else 0))
    dgate = pad.view(rows, -1, case["d"]).sum(1)
    dv = dx * gate
    dnv = dv * s["w_post"]
    dy = r_post * (dnv - v * (dnv * v).mean(1, keepdim=True))
    dt = s["x"].dtype
    return {"dx": dx.to(dt), "dy": dy.to(dt), "dgate": dgate.to(dt),
            "dw_post": (dv * v).sum(0), "dw_next": (dh * u).sum(0)}


def _plain_clip(case, s):
    sums = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]])
    norm = sums.sum().sqrt().float()
    coef = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    clipped = [(t.float() * coef).to(t.dtype) for t in s["grads"]]
    if "flat" in s:
        clipped = torch.cat([t.reshape(-1) for t in clipped])
    return {"norm": norm, "clipped": clipped}


def _plain_i8(case, s):
    E, k, o, most = case["E"], case["k"], case["n_out"], s["most"]
    j = torch.arange(most, device="cuda")
    real = j[None, :] < s["counts"][:, None]
    row = (s["starts"][:, None] + j[None, :]).clamp(max=s["rows"] - 1).long()
    x = s["x"][row].float()  # [E, most, k]
    scale = (x.abs().amax(-1).double() / 127).float()
    # a value next to the border of two steps needs the exact quotient
    q = (x.double() / scale[..., None].double()).round().nan_to_num(0.0).float()
    u = torch.bmm(q, s["w1"].float().transpose(1, 2)) * scale[..., None] * s["w1_scale"][:, None]
    if case["act"] == "swiglu":
        v = torch.bmm(q, s["w3"].float().transpose(1, 2))
        u = u * torch.sigmoid(u) * (v * scale[..., None] * s["w3_scale"][:, None])
    out = torch.zeros((s["rows"], o), dtype=s["x"].dtype, device="cuda")
    # rows behind a segment's last one go to a line that is cut off again
    to = torch.where(real, row, s["rows"])
    out = torch.cat([out, out[:1]])
    out[to.view(-1)] = u.to(out.dtype).view(-1, o)
    return out[:-1]


# --------------------------------------------------------------------------- the framework's calls
def _own_norm(case, s):
    from expert_dispatch_gemm_b200 import block
    if "cfg" not in s:
        s["cfg"] = block.norm_config(n=case["n"], d=case["d"], dtype=s["x"].dtype, eps=EPS,
                                     gate_tokens=case["gate_tokens"])
    block.moe_residual_norm_forward(s["cfg"], s["x"], s["y"], s["w_post"], s["gate"],
                                    s["w_next"], s["out"], s["h"], s["rstd_post"],
                                    s["rstd_next"])
    return {k: s[k] for k in ("out", "h", "rstd_post", "rstd_next")}


def _own_norm_backward(case, s):
    from expert_dispatch_gemm_b200 import block
    if "cfg" not in s:
        s["cfg"] = block.norm_config(n=case["n"], d=case["d"], dtype=s["x"].dtype, eps=EPS,
                                     gate_tokens=case["gate_tokens"])
        s["ws"] = block.norm_workspace(s["cfg"], "cuda")
    block.moe_residual_norm_backward(s["cfg"], s["dout"], s["dh"], s["x"], s["y"], s["w_post"],
                                     s["gate"], s["w_next"], s["rstd_post"], s["rstd_next"],
                                     s["dx"], s["dy"], s["dw_post"], s["dgate"], s["dw_next"],
                                     s["ws"])
    return {k: s[k] for k in ("dx", "dy", "dgate", "dw_post", "dw_next")}


def _own_clip(case, s):
    from expert_dispatch_gemm_b200 import block
    if "list" not in s:
        s["list"] = block.grad_list(s["grads"], s["clipped"])
        s["ws"] = block.grad_workspace(s["list"], "cuda")
        s["norm"] = torch.empty(2, dtype=torch.float32, device="cuda")
    block.moe_grad_clip(s["list"], case["max_norm"], s["norm"], s["ws"])
    return {"norm": s["norm"][0], "clipped": s["flat"] if "flat" in s else s["clipped"]}


def _own_i8(case, s):
    from expert_dispatch_gemm_b200 import block
    if "cfg" not in s:
        s["cfg"] = block.gemm_i8_config(groups=case["E"], rows=s["rows"], k=case["k"],
                                        n_out=case["n_out"], act=case["act"],
                                        dtype=s["x"].dtype)
        s["ws"] = block.gemm_i8_workspace(s["cfg"], "cuda")
    block.moe_quantize_rows(s["x"], s["q"], s["q_scale"], s["starts"], s["counts"])
    block.moe_gemm_i8(s["cfg"], s["q"], s["q_scale"], s["starts"], s["counts"], s["w1"],
                      s["w1_scale"], s.get("w3"), s.get("w3_scale"), s["out"], s["ws"])
    return s["out"]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        call = {"residual_norm": _own_norm, "residual_norm_backward": _own_norm_backward,
                "grad_clip": _own_clip, "gemm_i8": _own_i8}[op]
    else:
        call = {"residual_norm": _plain_norm, "residual_norm_backward": _plain_norm_backward,
                "grad_clip": _plain_clip, "gemm_i8": _plain_i8}[op]
    return call(case, state)


# --------------------------------------------------------------------------- work
def work(case):
    if case["op"] in ("residual_norm", "residual_norm_backward"):
        n, d, b = case["n"], case["d"], 4 if case["dtype"] == "f32" else 2
        gate = _gate_rows(case) * d * b
        if case["op"] == "residual_norm":  # x, y in; out, h out
            stats = 8 * n if case["stats"] else 0
            return {"bytes": 4 * n * d * b + gate + 8 * d + stats, "flops": 12 * n * d}
        # dout, dh, out, y, both inverse norms in; dx, dy and the weights' out
        return {"bytes": 6 * n * d * b + 2 * gate + 16 * d + 8 * n, "flops": 26 * n * d}
    if case["op"] == "grad_clip":
        b = 4 if case["dtype"] == "f32" else 2
        shapes = _shapes(case)
        total = sum(math.prod(s) * (4 if r else b) for s, r in shapes)
        return {"bytes": 2 * total + 4, "flops": 3 * sum(math.prod(s) for s, _ in shapes)}
    b = 4 if case["dtype"] == "f32" else 2
    E, k, o, rows = case["E"], case["k"], case["n_out"], case["rows"]
    sides = 2 if case["act"] == "swiglu" else 1
    experts = min(E, rows)  # experts that can have a row
    return {"bytes": rows * (k + o) * b + sides * experts * o * (k + 4) + 8 * E,
            "flops": 2 * rows * k * o * sides}


# --------------------------------------------------------------------------- the definition in 64 bits
def _exact_norm(case, s):
    f = {k: s[k].double() for k in ("x", "y", "w_post", "w_next", "gate")}
    token = torch.arange(case["n"], device="cuda")
    gate = f["gate"][token // case["gate_tokens"] if case["gate_tokens"] else token * 0]
    r1 = 1 / torch.sqrt((f["y"] ** 2).sum(1) / case["d"] + EPS)
    out = f["x"] + gate * f["w_post"] * f["y"] * r1[:, None]
    r2 = 1 / torch.sqrt((out ** 2).sum(1) / case["d"] + EPS)
    h = out * r2[:, None] * f["w_next"]
    stats = case["stats"]
    return {"out": out, "h": h, "rstd_post": r1 if stats else None,
            "rstd_next": r2 if stats else None}


def _exact_norm_backward(case, s):
    """The same gradients from the Jacobian of each norm: d(r v)/dv = r (I - (r v)(r v)^T / d)."""
    f = {k: s[k].double() for k in ("x", "y", "w_post", "w_next", "gate", "dout", "dh",
                                     "rstd_post", "rstd_next")}
    d = case["d"]
    token = torch.arange(case["n"], device="cuda")
    which = token // case["gate_tokens"] if case["gate_tokens"] else token * 0
    gate = f["gate"][which]
    r1, r2 = f["rstd_post"].unsqueeze(1), f["rstd_next"].unsqueeze(1)
    a = f["dh"] * f["w_next"]
    inner = torch.einsum("td,td->t", a, f["x"]).unsqueeze(1)
    dx = f["dout"] + r2 * a - f["x"] * inner * r2 ** 3 / d
    b = dx * gate * f["w_post"]
    inner = torch.einsum("td,td->t", b, f["y"]).unsqueeze(1)
    dy = r1 * b - f["y"] * inner * r1 ** 3 / d
    share = dx * f["w_post"] * f["y"] * r1
    dgate = torch.zeros_like(f["gate"]).index_add_(0, which, share)
    ones = torch.ones(case["n"], dtype=torch.float64, device="cuda")
    return {"dx": dx, "dy": dy, "dgate": dgate, "dw_post": ones @ (dx * gate * f["y"] * r1),
            "dw_next": ones @ (f["dh"] * f["x"] * r2)}


def _exact_clip(case, s):
    total = 0.0
    for t in s["grads"]:
        total += float(torch.linalg.vector_norm(t.double())) ** 2
    norm = math.sqrt(total)
    factor = min(1.0, case["max_norm"] / (norm + 1e-6))
    clipped = [t.double() * factor for t in s["grads"]]
    if "flat" in s:
        clipped = torch.cat([t.flatten() for t in clipped])
    return {"norm": torch.tensor(norm, dtype=torch.float64), "clipped": clipped}


def _exact_i8(case, s):
    out = torch.zeros((s["rows"], case["n_out"]), dtype=torch.float64, device="cuda")
    for e, (first, count) in enumerate(zip(s["starts"].tolist(), s["counts"].tolist())):
        if count == 0:
            continue
        x = s["x"][first:first + count].double()
        # the scale is a 32-bit number: the largest magnitude of the row over 127
        step = (x.abs().max(1, keepdim=True).values / 127).float().double()
        q = torch.where(step > 0, torch.round(x / torch.where(step > 0, step, 1.0)), 0.0)
        sides = [(q @ s[w][e].double().T) * step * s[w + "_scale"][e].double()
                 for w in ("w1", "w3") if w in s]
        out[first:first + count] = (sides[0] if len(sides) == 1 else
                                    sides[0] / (1 + torch.exp(-sides[0])) * sides[1])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    f = {"residual_norm": _exact_norm, "residual_norm_backward": _exact_norm_backward,
         "grad_clip": _exact_clip, "gemm_i8": _exact_i8}[case["op"]]
    return f(case, s)
