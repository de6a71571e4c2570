"""The training operators around the compressor, as a user's program calls them, and what they have to do.

Four families: layer norm (``norm_forward``, ``norm_backward``), a gated linear recurrence
(``recurrence_forward``, and ``recurrence_train``, which is forward and backward), the norm of many gradients
with its clipping coefficient (``grad_norm``), and an AdamW step over many tensors with its moments in 32 or
in 8 bits (``adamw``). ``run`` computes them with elementary torch operations in 32 bits, or, where
``own`` is true, with this repository's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

#: Elements that share one scale of the 8-bit moments; flat buffers give every tensor a multiple of it.
BLOCK = 256
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.01, 200
NORM_EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decoder of width 2048 as it is served: latency alone
        {"name": "norm_forward 1x2048", "op": "norm_forward", "rows": 1, "dim": 2048, "x": "bf16", "w": "bf16"},
        # the activations of 8 sequences of 2048 tokens at that width: a training step's forward pass
        {"name": "norm_forward 16384x2048", "op": "norm_forward", "rows": 16384, "dim": 2048, "x": "bf16", "w": "f32"},
        # and its backward pass, with the gradients of the weight and the bias
        {"name": "norm_backward 16384x2048", "op": "norm_backward", "rows": 16384, "dim": 2048, "x": "bf16",
         "w": "f32"},
        # an odd width in 32 bits, with a number of rows that no tile divides
        {"name": "norm_backward 3001x1001", "op": "norm_backward", "rows": 3001, "dim": 1001, "x": "f32", "w": "f32"},
        # one new token for each of 64 sequences that are being generated
        {"name": "recurrence_forward 64x1x1024", "op": "recurrence_forward", "batch": 64, "steps": 1, "dim": 1024,
         "x": "bf16", "ragged": False},
        # a recurrent layer's training step on 16 sequences of 2048 tokens, width 1024
        {"name": "recurrence_train 16x2048x1024", "op": "recurrence_train", "batch": 16, "steps": 2048, "dim": 1024,
         "x": "bf16", "ragged": False},
        # few, long and ragged sequences (one of them empty) of a width that no warp divides, in 32 bits
        {"name": "recurrence_train 4x20011x501", "op": "recurrence_train", "batch": 4, "steps": 20011, "dim": 501,
         "x": "f32", "ragged": True},
        # the gradients of a small fully connected layer, and of a 1.3B decoder
        {"name": "grad_norm fc", "op": "grad_norm", "tensors": "fc", "g": "f32"},
        {"name": "grad_norm decoder", "op": "grad_norm", "tensors": "decoder", "g": "bf16"},
        # the step over that small layer, over a net of LSTM and wide layers, and over the decoder with 8-bit moments
        {"name": "adamw32 fc", "op": "adamw", "tensors": "fc", "w": "f32", "g": "f32", "bits": 32},
        {"name": "adamw32 lstm", "op": "adamw", "tensors": "lstm", "w": "f32", "g": "f32", "bits": 32},
        {"name": "adamw8 decoder", "op": "adamw", "tensors": "decoder", "w": "f32", "g": "bf16", "bits": 8},
    ]


def draw(rng):
    def spread(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    op = rng.choice(["norm_forward", "norm_backward", "recurrence_forward", "recurrence_train", "grad_norm", "adamw"])
    if op.startswith("norm"):
        dim = spread(1, 16384)
        return {"op": op, "rows": spread(1, min(65536, (1 << 26) // dim)), "dim": dim, "x": rng.choice(["f32", "bf16"]),
                "w": rng.choice(["f32", "bf16"])}
    if op.startswith("recurrence"):
        dim = spread(1, 4096)
        steps = spread(1, 32768)
        batch = spread(1, max(1, min(256, (1 << 25) // (dim * steps))))
        return {"op": op, "batch": batch, "steps": steps, "dim": dim, "x": rng.choice(["f32", "bf16"]),
                "ragged": rng.random() < 0.5}
    case = {"op": op, "tensors": "random", "count": spread(1, 600), "most": spread(16, 1 << 22),
            "sizes": rng.randrange(1 << 30), "g": rng.choice(["f32", "bf16"])}
    if op == "adamw":
        case.update(w=rng.choice(["f32", "bf16"]), bits=rng.choice([8, 32]))
    return case


def sizes_of(case):
    """Elements of each tensor, and whether it is a matrix (which decays)."""
    kind = case["tensors"]
    if kind == "fc":
        return [(500 * 800, True), (800, False)]
    if kind == "lstm":
        return [(4 * 1024 * 2048, True)] * 4 + [(4096 * 4096, True)] * 6
    if kind == "decoder":
        d, ffn, vocab, ctx = 2048, 8192, 50304, 2048
        block = [(d, False), (d, False), (3 * d * d, True), (3 * d, False), (d * d, True), (d, False),
                 (d, False), (d, False), (ffn * d, True), (ffn, False), (d * ffn, True), (d, False)]
        return [(vocab * d, True), (ctx * d, True)] + block * 24 + [(d, False), (d, False)]
    r = random.Random(case["sizes"])
    return [(max(1, int(math.exp(r.uniform(0.0, math.log(case["most"]))))), r.random() < 0.7)
            for _ in range(case["count"])]


def lengths_of(case):
    """The sequences' lengths: all of them whole, or spread from none to all of the steps."""
    batch, steps = case["batch"], case["steps"]
    if not case["ragged"]:
        return [steps] * batch
    return [steps - int(steps * ((0.618034 * b) % 1.0)) if b != 1 else 0 for b in range(batch)]


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        n, d, e, ew = case["rows"] * case["dim"], case["dim"], BYTES[case["x"]], BYTES[case["w"]]
        if op == "norm_forward":
            return {"bytes": 2 * n * e + 2 * d * ew + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 3 * d * ew + 8 * case["rows"], "flops": 14 * n}
    if op.startswith("recurrence"):
        d, e = case["dim"], BYTES[case["x"]]
        valid, whole = sum(lengths_of(case)) * d, case["batch"] * case["steps"] * d
        ends = 8 * case["batch"] * d
        if op == "recurrence_forward":
            return {"bytes": e * (2 * valid + whole) + ends, "flops": 8 * valid}
        return {"bytes": e * (5 * valid + 3 * whole) + 2 * ends, "flops": 28 * valid}
    n = sum(s for s, _ in sizes_of(case))
    if op == "grad_norm":
        return {"bytes": BYTES[case["g"]] * n + 8, "flops": 2 * n}
    blocks = sum(-(-s // BLOCK) for s, _ in sizes_of(case))
    state = 16 * n if case["bits"] == 32 else 4 * n + 16 * blocks
    return {"bytes": (2 * BYTES[case["w"]] + BYTES[case["g"]]) * n + state, "flops": 16 * n}


# --------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _norm_inputs(case, seed):
    gen, dt, wt = _generator(seed), DTYPES[case["x"]], DTYPES[case["w"]]
    rows, dim = case["rows"], case["dim"]
    # a residual stream: channels of unlike scale, and an offset that differs from row to row
    x = (_normal(gen, rows, dim) * (1 + _normal(gen, dim).abs()) + 0.5 * _normal(gen, rows, 1)).to(dt)
    s = {"x": x, "w": (1 + 0.2 * _normal(gen, dim)).to(wt), "b": (0.1 * _normal(gen, dim)).to(wt)}
    if case["op"] == "norm_backward":
        s["dy"] = (0.01 * _normal(gen, rows, dim)).to(dt)
        wide = x.float()
        s["mean"] = wide.mean(1)
        s["rstd"] = 1.0 / torch.sqrt((wide - s["mean"][:, None]).square().mean(1) + NORM_EPS)
    return s


def _recurrence_inputs(case, seed):
    gen, dt = _generator(seed), DTYPES[case["x"]]
    batch, steps, dim = case["batch"], case["steps"], case["dim"]
    zx = _normal(gen, batch, steps, 2 * dim)
    zx[..., :dim] += 2.0  # a forget gate starts out open: most of the state is kept
    s = {"zx": zx.to(dt), "h0": _normal(gen, batch, dim)}
    s["lengths"] = torch.tensor(lengths_of(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
    if case["op"] == "recurrence_train":
        s["dy"] = (0.01 * _normal(gen, batch, steps, dim)).to(dt)
        s["dh_last"] = 0.01 * _normal(gen, batch, dim)
    return s


def _offsets(case):
    """Where each tensor starts in a flat buffer, and the buffer's length."""
    padded = np.array([0] + [-(-s // BLOCK) * BLOCK for s, _ in sizes_of(case)], dtype=np.int64)
    ends = np.cumsum(padded)
    return ends[:-1].tolist(), int(ends[-1])


def _views(flat, case):
    return [flat[o:o + s] for o, (s, _) in zip(_offsets(case)[0], sizes_of(case))]


def _inside(case, total):
    """Which elements of the flat buffer belong to a tensor."""
    offsets = torch.tensor(_offsets(case)[0], device="cuda")
    sizes = torch.tensor([s for s, _ in sizes_of(case)], device="cuda")
    starts = torch.arange(0, total, BLOCK, device="cuda")
    owner = torch.searchsorted(offsets, starts, right=True) - 1
    left = (sizes[owner] - (starts - offsets[owner])).clamp(0, BLOCK)
    return torch.arange(BLOCK, device="cuda")[None, :] < left[:, None], owner


def _to_eight(values, at_least_one):
    """Blocks of values as e4m3 numbers and the scale of each block."""
    top = values.abs().amax(1, keepdim=True)
    used = ~(top < 2.0 ** -96)
    most = torch.full_like(top, 448.0)  # a tensor: torch divides by, or into, a number through a reciprocal
    scale = torch.where(used, top / most, 0.0)
    inverse = torch.where(used, most / top, 0.0)
    code = (values * inverse).to(torch.float8_e4m3fn)
    if at_least_one:
        code = torch.where((values > 0) & (code.float() == 0), 2.0 ** -9, code.float()).to(torch.float8_e4m3fn)
    return code, scale


def _tensor_inputs(case, seed):
    gen = _generator(seed)
    total = _offsets(case)[1]
    inside, owner = _inside(case, total)
    s = {}
    g = _normal(gen, total // BLOCK, BLOCK).mul_(1e-3).mul_(inside)
    s["g"] = g.to(DTYPES[case["g"]]).view(-1)
    if case["op"] == "adamw":
        s["w"] = _normal(gen, total // BLOCK, BLOCK).mul_(0.02).mul_(inside).to(DTYPES[case["w"]]).view(-1)
        # the moments in the middle of a run: some steps' worth of averaged gradients
        m = _normal(gen, total // BLOCK, BLOCK).mul_(2.5e-4).mul_(inside)
        u = _normal(gen, total // BLOCK, BLOCK).mul_(0.2).add_(1.0).abs_().mul_(1e-3).mul_(inside)
        if case["bits"] == 8:
            s["m"], s["m_scale"] = (t.view(-1) for t in _to_eight(m, False))
            s["v"], s["v_scale"] = (t.view(-1) for t in _to_eight(u, True))
        else:
            s["m"], s["v"] = m.view(-1), u.square_().view(-1)
        decays = np.array([DECAY if matrix else 0.0 for _, matrix in sizes_of(case)], dtype=np.float32)
        kept = (1.0 - float(np.float32(LR)) * decays.astype(np.float64)).astype(np.float32)
        s["kept"] = torch.from_numpy(kept).cuda()[owner][:, None]  # 1 - lr * decay, by block
        s["decays"] = decays.tolist()
    return s


def prepare(case, seed):
    op = case["op"]
    s = {"norm": _norm_inputs, "recurrence": _recurrence_inputs}.get(op.split("_")[0], _tensor_inputs)(case, seed)
    s["case"] = case
    if own:
        s["plan"] = _plan(s)
    return s


# ---------------------------------------------------------------------------- plain forms

def _norm_forward(s):
    x = s["x"].float()
    mean = x.mean(1)
    centred = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(centred.square().mean(1) + NORM_EPS)
    y = centred * rstd[:, None] * s["w"].float() + s["b"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _norm_backward(s):
    dy, w = s["dy"].float(), s["w"].float()
    normed = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - normed * (g * normed).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * normed).sum(0).to(s["w"].dtype), "db": dy.sum(0).to(s["w"].dtype)}


def _prefix(a, h):
    """h_t + a_t h_{t-1} + a_t a_{t-1} h_{t-2} + ... along the steps, by doubling."""
    reach, steps = 1, h.shape[1]
    while reach < steps:
        h = torch.cat([h[:, :reach], h[:, reach:] + a[:, reach:] * h[:, :-reach]], 1)
        a = torch.cat([a[:, :reach], a[:, reach:] * a[:, :-reach]], 1)
        reach *= 2
    return h


def _recurrence_parts(s):
    dim = s["zx"].shape[2] // 2
    z, x = s["zx"][..., :dim].float(), s["zx"][..., dim:].float()
    keep = torch.sigmoid(z)
    take = torch.sigmoid(-z)
    if s["lengths"] is None:
        live = torch.ones((), dtype=torch.bool, device=z.device)
    else:
        live = (torch.arange(z.shape[1], device=z.device)[None, :] < s["lengths"][:, None])[..., None]
    a = torch.where(live, keep, 1.0)
    add = torch.where(live, take * x, 0.0)
    add = torch.cat([add[:, :1] + a[:, :1] * s["h0"][:, None], add[:, 1:]], 1)
    return x, keep, take, live, a, _prefix(a, add)


def _recurrence_forward(s):
    _, _, _, live, _, h = _recurrence_parts(s)
    return {"y": torch.where(live, h, 0.0).to(s["zx"].dtype), "h_last": h[:, -1].clone()}


def _recurrence_train(s):
    x, keep, take, live, a, h = _recurrence_parts(s)
    dh = torch.where(live, s["dy"].float(), 0.0)
    dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dh_last"][:, None]], 1).flip(1)
    after = torch.cat([torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
    g = _prefix(after, dh).flip(1)
    before = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
    dz = torch.where(live, g * keep * take * (before - x), 0.0)
    dx = torch.where(live, g * take, 0.0)
    return {"y": torch.where(live, h, 0.0).to(s["zx"].dtype), "h_last": h[:, -1].clone(),
            "dzx": torch.cat([dz, dx], 2).to(s["zx"].dtype), "dh0": a[:, 0] * g[:, 0]}


def _grad_norm(s):
    norm = torch.sqrt(s["g"].float().square().sum())
    return torch.stack([norm, torch.clamp(1.0 / (norm + 1e-6), max=1.0)])


def _adamw_numbers():
    """The step's constants, each rounded once to 32 bits."""
    one, f = np.float32(1.0), np.float32
    c1, c2 = f(1.0 - BETA1 ** STEP), f(1.0 - BETA2 ** STEP)
    return {"beta1": float(f(BETA1)), "beta2": float(f(BETA2)), "rest1": float(one - f(BETA1)),
            "rest2": float(one - f(BETA2)), "step": float(f(float(f(LR)) / float(c1))),
            "root": float(f(1.0 / math.sqrt(float(c2)))), "eps": float(f(EPS)), "c1": float(c1), "c2": float(c2)}


def _adamw(s):
    k, eight = _adamw_numbers(), s["case"]["bits"] == 8
    w, g = s["w"].view(-1, BLOCK).float(), s["g"].view(-1, BLOCK).float()
    m, v = s["m"].view(-1, BLOCK).float(), s["v"].view(-1, BLOCK).float()
    if eight:
        m = m * s["m_scale"][:, None]
        v = (v * s["v_scale"][:, None]).square()
    m = k["beta1"] * m + k["rest1"] * g
    v = k["beta2"] * v + k["rest2"] * (g * g)
    u = torch.sqrt(v)
    w = s["kept"] * w - k["step"] * (m / (u * k["root"] + k["eps"]))
    s["w"].copy_(w.view(-1))
    if not eight:
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
        return {"w": s["w"], "m": s["m"], "v": s["v"]}
    for name, values in (("m", m), ("v", u)):
        code, scale = _to_eight(values, name == "v")
        s[name].copy_(code.view(-1))
        s[name + "_scale"].copy_(scale.view(-1))
    return {"w": s["w"], "m": s["m"], "v": s["v"], "m_scale": s["m_scale"], "v_scale": s["v_scale"]}


# ------------------------------------------------------------------- the framework's calls

def _code(dtype):
    import residual_gradient_compression_gb300 as ac
    return ac.BF16 if dtype == "bf16" else ac.F32


def _zeros(nbytes):
    return torch.zeros(max(16, nbytes), dtype=torch.uint8, device="cuda")


def _plan(s):
    """Handles, outputs and workspaces, as a program makes them before its first step."""
    import residual_gradient_compression_gb300 as ac
    case, p = s["case"], {"ac": ac}
    op = case["op"]
    if op.startswith("norm"):
        p["h"] = ac.adacomp_layer_norm_init(case["dim"], _code(case["x"]), _code(case["w"]), NORM_EPS)
        if op == "norm_forward":
            p["y"] = torch.empty_like(s["x"])
            p["mean"], p["rstd"] = (torch.empty(case["rows"], device="cuda") for _ in range(2))
        else:
            p["dx"], p["dw"], p["db"] = (torch.empty_like(s[k]) for k in ("x", "w", "b"))
            p["ws"] = _zeros(ac.adacomp_layer_norm_backward_ws_bytes(p["h"], case["rows"]))
    elif op.startswith("recurrence"):
        d = case["dim"]
        p["h"] = ac.adacomp_recurrence_init(d, _code(case["x"]))
        p["z"], p["x"] = s["zx"][..., :d], s["zx"][..., d:]
        p["y"] = torch.empty(case["batch"], case["steps"], d, dtype=s["zx"].dtype, device="cuda")
        p["h_last"] = torch.empty_like(s["h0"])
        p["carry"] = None
        if op == "recurrence_train":
            carry = ac.adacomp_recurrence_carry_bytes(p["h"], case["batch"], case["steps"])
            p["carry"] = torch.empty(carry // 4, device="cuda")
            p["dzx"] = torch.empty_like(s["zx"])
            p["dz"], p["dx"] = p["dzx"][..., :d], p["dzx"][..., d:]
            p["dh0"] = torch.empty_like(s["h0"])
    else:
        sizes = [n for n, _ in sizes_of(case)]
        p["h"] = ac.adacomp_adamw_init(sizes, [_code(case.get("w", "f32"))] * len(sizes),
                                       [_code(case["g"])] * len(sizes), s.get("decays", [0.0] * len(sizes)),
                                       case.get("bits", 32))
        p["g"] = ac.adacomp_pointers(_views(s["g"], case))
        if op == "grad_norm":
            p["result"] = torch.empty(2, device="cuda")
            p["ws"] = _zeros(p["h"].norm_ws_bytes)
        else:
            p["w"], p["m"], p["v"] = (ac.adacomp_pointers(_views(s[k], case)) for k in ("w", "m", "v"))
            if case["bits"] == 8:
                at = [o // BLOCK for o in _offsets(case)[0]]
                for k in ("m_scale", "v_scale"):
                    p[k] = ac.adacomp_pointers([s[k][o:o + -(-n // BLOCK)] for o, n in zip(at, sizes)])
    return p


def _own(s):
    p, case = s["plan"], s["case"]
    ac, h, op = p["ac"], p["h"], s["case"]["op"]
    if op == "norm_forward":
        ac.adacomp_layer_norm_forward(h, s["x"], s["w"], s["b"], p["y"], p["mean"], p["rstd"])
        return {"y": p["y"], "mean": p["mean"], "rstd": p["rstd"]}
    if op == "norm_backward":
        ac.adacomp_layer_norm_backward(h, s["dy"], s["x"], s["w"], s["mean"], s["rstd"], p["dx"], p["dw"], p["db"],
                                       p["ws"])
        return {"dx": p["dx"], "dw": p["dw"], "db": p["db"]}
    if op.startswith("recurrence"):
        ac.adacomp_recurrence_forward(h, p["z"], p["x"], p["y"], h0=s["h0"], lengths=s["lengths"],
                                      h_last=p["h_last"], carry=p["carry"])
        if op == "recurrence_forward":
            return {"y": p["y"], "h_last": p["h_last"]}
        ac.adacomp_recurrence_backward(h, p["z"], p["x"], s["dy"], p["carry"], p["dz"], p["dx"], lengths=s["lengths"],
                                       dh_last=s["dh_last"], dh0=p["dh0"])
        return {"y": p["y"], "h_last": p["h_last"], "dzx": p["dzx"], "dh0": p["dh0"]}
    if op == "grad_norm":
        ac.adacomp_grad_norm(h, p["g"], p["result"], p["ws"], max_norm=1.0)
        return p["result"]
    k = _adamw_numbers()
    ac.adacomp_adamw_step(h, p["w"], p["g"], p["m"], p["v"], LR, BETA1, BETA2, EPS, k["c1"], k["c2"],
                          m_scale=p.get("m_scale"), v_scale=p.get("v_scale"))
    names = ("w", "m", "v", "m_scale", "v_scale") if case["bits"] == 8 else ("w", "m", "v")
    return {n: s[n] for n in names}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"norm_forward": _norm_forward, "norm_backward": _norm_backward, "recurrence_forward": _recurrence_forward,
            "recurrence_train": _recurrence_train, "grad_norm": _grad_norm, "adamw": _adamw}[op](state)


# --------------------------------------------------------------------------- in 64 bits

def _exact_norm(s):
    x, w = s["x"].double(), s["w"].double()
    n = x.shape[1]
    if "dy" not in s:
        mean = x.sum(1) / n
        var = ((x - mean[:, None]) ** 2).sum(1) / n
        rstd = (var + NORM_EPS) ** -0.5
        return {"y": (x - mean[:, None]) * (rstd[:, None] * w) + s["b"].double(), "mean": mean, "rstd": rstd}
    dy, mean, rstd = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
    xh = rstd * (x - mean)
    dxh = dy * w
    dx = (rstd / n) * (n * dxh - dxh.sum(1, keepdim=True) - xh * (dxh * xh).sum(1, keepdim=True))
    return {"dx": dx, "dw": (xh * dy).sum(0), "db": dy.sum(0)}


def _exact_recurrence(s, train):
    """The recurrence step by step, as it is written."""
    dim, steps = s["zx"].shape[2] // 2, s["zx"].shape[1]
    z, x = s["zx"][..., :dim].double(), s["zx"][..., dim:].double()
    a = 1 / (1 + torch.exp(-z))
    b = 1 / (1 + torch.exp(z))
    count = torch.full((z.shape[0],), steps, device=z.device) if s["lengths"] is None else s["lengths"]
    hs = torch.zeros_like(z)
    before = torch.zeros_like(z)
    h = s["h0"].double()
    for t in range(steps):
        on = (t < count)[:, None]
        before[:, t] = h
        h = torch.where(on, a[:, t] * h + b[:, t] * x[:, t], h)
        hs[:, t] = h * on
    out = {"y": hs, "h_last": h}
    if train:
        dz, dx = torch.zeros_like(z), torch.zeros_like(z)
        dh = s["dh_last"].double()
        for t in range(steps - 1, -1, -1):
            on = (t < count)[:, None]
            g = torch.where(on, dh + s["dy"][:, t].double(), dh)
            dz[:, t] = g * (before[:, t] - x[:, t]) * a[:, t] * b[:, t] * on
            dx[:, t] = g * b[:, t] * on
            dh = torch.where(on, a[:, t] * g, g)
        out["dzx"], out["dh0"] = torch.cat([dz, dx], 2), dh
    return out


def _exact_eight(v, floor):
    """Values in e4m3 with 3 bits after the point, from their definition; and the scale."""
    top = v.abs().amax(1, keepdim=True)
    r = torch.where(top > 0, v * 448 / top, torch.zeros_like(v))
    e = torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6)))
    q = torch.exp2(e - 3)
    r = torch.round(r / q) * q
    if floor:
        r = torch.where((v > 0) & (r == 0), torch.full_like(r, 2.0 ** -9), r)
    return r.view(-1), (top / 448).view(-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        return _exact_norm(s)
    if op.startswith("recurrence"):
        return _exact_recurrence(s, op == "recurrence_train")
    if op == "grad_norm":
        n = math.sqrt(sum(float((c.double() ** 2).sum()) for c in s["g"].split(1 << 26)))
        return torch.tensor([n, min(1.0, 1.0 / (n + 1e-6))], dtype=torch.float64)
    rows, parts = 1 << 18, []
    for i in range(0, s["w"].numel() // BLOCK, rows):
        w, g, m, v = (s[k].view(-1, BLOCK)[i:i + rows].to(torch.float32).double() for k in ("w", "g", "m", "v"))
        if case["bits"] == 8:
            m = m * s["m_scale"][i:i + rows, None].double()
            v = (v * s["v_scale"][i:i + rows, None].double()) ** 2
        m = m + (1 - BETA1) * (g - m)
        v = v + (1 - BETA2) * (g ** 2 - v)
        hat_m, hat_v = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
        w = w * s["kept"][i:i + rows].double() - LR * hat_m / (hat_v ** 0.5 + EPS)
        part = {"w": w.view(-1), "m": m.view(-1), "v": v.view(-1)}
        if case["bits"] == 8:
            part["m"], part["m_scale"] = _exact_eight(m, False)
            part["v"], part["v_scale"] = _exact_eight(v ** 0.5, True)
        parts.append(part)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
