"""Matrix products with an epilogue, and losses over a large vocabulary, as a user's program calls them, and what
they have to do.

Three families: a linear layer with bias, activation and residual in one call (``linear_forward``, and
``linear_train``, which is forward and backward), softmax cross entropy straight from the hidden states and the
vocabulary's weights (``vocab_forward``, ``vocab_train``), and distillation from a teacher's top logits over the same
vocabulary (``distill_forward``, ``distill_train``). ``run`` computes them with elementary torch operations in 32 bits,
or, where ``own`` is true, with this repository's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
ACTIVATIONS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token through the wide layer of a decoder's block of width 2048: latency alone
        {"name": "linear_forward 1x2048x8192", "op": "linear_forward", "rows": 1, "din": 2048, "dout": 8192, "x": "bf16",
         "act": "gelu", "bias": True, "residual": False},
        # 64 sequences that are being generated, through the layer back to that width, onto the residual stream
        {"name": "linear_forward 64x8192x2048", "op": "linear_forward", "rows": 64, "din": 8192, "dout": 2048,
         "x": "bf16", "act": "none", "bias": True, "residual": True},
        # a training step's wide layer, on 8 sequences of 2048 tokens
        {"name": "linear_train 16384x2048x8192", "op": "linear_train", "rows": 16384, "din": 2048, "dout": 8192,
         "x": "bf16", "act": "gelu", "bias": True, "residual": False},
        # a small fully connected layer's step, a batch of 64 in 32 bits
        {"name": "linear_train 64x800x500", "op": "linear_train", "rows": 64, "din": 800, "dout": 500, "x": "f32",
         "act": "relu", "bias": True, "residual": False},
        # odd sizes in 32 bits that no tile divides, with everything in the epilogue
        {"name": "linear_train 3001x1001x777", "op": "linear_train", "rows": 3001, "din": 1001, "dout": 777, "x": "f32",
         "act": "silu", "bias": True, "residual": True},
        # the likelihood of a few tokens: the vocabulary's weights are read for 32 rows
        {"name": "vocab_forward 32x2048x50304", "op": "vocab_forward", "rows": 32, "dim": 2048, "vocab": 50304,
         "x": "bf16", "ignored": 0.0},
        # the loss of 4 sequences of 2048 tokens, with its gradients: pretraining, every token counts
        {"name": "vocab_train 8192x2048x50304", "op": "vocab_train", "rows": 8192, "dim": 2048, "vocab": 50304,
         "x": "bf16", "ignored": 0.0},
        # fine-tuning: half of the tokens are prompts or padding, and have no loss
        {"name": "vocab_train half 4096x2048x50304", "op": "vocab_train", "rows": 4096, "dim": 2048, "vocab": 50304,
         "x": "bf16", "ignored": 0.5},
        # odd sizes in 32 bits, a small vocabulary, some rows without a target
        {"name": "vocab_train 2003x501x10007", "op": "vocab_train", "rows": 2003, "dim": 501, "vocab": 10007, "x": "f32",
         "ignored": 0.1},
        # how far a student is from its teacher, on a small batch
        {"name": "distill_forward 512x2048x50304", "op": "distill_forward", "rows": 512, "dim": 2048, "vocab": 50304,
         "x": "bf16", "k": 64, "temperature": 1.0, "ignored": 0.0},
        # a student's training step from the 64 largest logits of every token
        {"name": "distill_train 4096x2048x50304", "op": "distill_train", "rows": 4096, "dim": 2048, "vocab": 50304,
         "x": "bf16", "k": 64, "temperature": 2.0, "ignored": 0.0},
        # odd sizes in 32 bits; lists of unlike lengths, some rows with none
        {"name": "distill_train 999x641x8191", "op": "distill_train", "rows": 999, "dim": 641, "vocab": 8191, "x": "f32",
         "k": 20, "temperature": 1.5, "ignored": 0.2},
    ]


def draw(rng):
    def spread(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    op = rng.choice(["linear_forward", "linear_train", "vocab_forward", "vocab_train", "distill_forward", "distill_train"])
    x = rng.choice(["f32", "bf16"])
    most = 1 << 38 if x == "bf16" else 1 << 36  # products: rows x inputs x outputs
    if op.startswith("linear"):
        din, dout = spread(1, 8192), spread(1, 8192)
        return {"op": op, "rows": spread(1, min(16384, most // (din * dout))), "din": din, "dout": dout, "x": x,
                "act": rng.choice(ACTIVATIONS), "bias": rng.random() < 0.7, "residual": rng.random() < 0.4}
    dim, vocab = spread(8, 2048), spread(100, 65536)
    case = {"op": op, "rows": spread(1, min(8192, most // (dim * vocab))), "dim": dim, "vocab": vocab, "x": x,
            "ignored": rng.choice([0.0, rng.uniform(0.0, 0.9)])}
    if op.startswith("distill"):
        case.update(k=min(vocab, spread(1, 128)), temperature=rng.choice([1.0, rng.uniform(0.5, 4.0)]))
    return case


def is_valid(case):
    """Which rows have a loss: the others are spread over the rows, as prompts and padding are."""
    return [((0.618034 * (r + 1)) % 1.0) >= case["ignored"] for r in range(case["rows"])]


def work(case):
    op, e, rows = case["op"], BYTES[case["x"]], case["rows"]
    if op.startswith("linear"):
        din, dout = case["din"], case["dout"]
        weights = din * dout + (dout if case["bias"] else 0)
        products = 2 * rows * din * dout
        forward = rows * (din + dout * (2 if case["residual"] else 1)) + weights
        if op == "linear_forward":
            return {"bytes": e * forward, "flops": products}
        # dy is read, and dx, dw and db are written; the value before the activation is an output too
        backward = rows * (dout + din) + weights + (0 if case["act"] == "none" else rows * dout)
        return {"bytes": e * (forward + backward), "flops": 3 * products}
    dim, vocab, valid = case["dim"], case["vocab"], sum(is_valid(case))
    lists = rows * (8 * case["k"] if op.startswith("distill") else 8)
    nbytes = e * (valid * dim + vocab * dim) + lists + 8 * rows
    if op.endswith("forward"):
        return {"bytes": nbytes, "flops": 2 * valid * dim * vocab}
    return {"bytes": nbytes + e * (rows * dim + vocab * dim) + 4 * rows, "flops": 6 * valid * dim * vocab}


# --------------------------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _linear_inputs(case, gen):
    dt, rows, din, dout = DTYPES[case["x"]], case["rows"], case["din"], case["dout"]
    s = {"x": _normal(gen, rows, din).to(dt), "w": (_normal(gen, dout, din) * din ** -0.5).to(dt)}
    s["b"] = (0.1 * _normal(gen, dout)).to(dt) if case["bias"] else None
    s["r"] = _normal(gen, rows, dout).to(dt) if case["residual"] else None
    if case["op"] == "linear_train":
        s["dy"] = (0.01 * _normal(gen, rows, dout)).to(dt)
    return s


def _head_inputs(case, gen):
    dt, rows, dim, vocab = DTYPES[case["x"]], case["rows"], case["dim"], case["vocab"]
    w = _normal(gen, vocab, dim) * (2.0 * dim ** -0.5)
    liked = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    # hidden states out of a norm, which lean towards a token: some rows are sure of it, some are not
    lean = 4.0 * torch.rand(rows, 1, generator=gen, device="cuda")
    x = _normal(gen, rows, dim) + lean * w[liked] * 0.5
    valid = torch.tensor(is_valid(case), device="cuda")
    s = {"x": x.to(dt), "w": w.to(dt)}
    if case["op"].startswith("vocab"):
        s["target"] = torch.where(valid, liked, -100)
    else:
        k = case["k"]
        # k different tokens, the liked one among them, with the logits of a teacher that likes it most
        step = 1 + (torch.rand(rows, 1, generator=gen, device="cuda") * (vocab // k)).long().clamp(max=vocab // k - 1)
        index = (liked[:, None] + torch.arange(k, device="cuda") * step) % vocab
        fall = -torch.log(torch.rand(rows, k, generator=gen, device="cuda").clamp(min=1e-6))
        fall[:, 0] = 0.0
        s["logit"] = 12.0 + _normal(gen, rows, 1) - torch.cumsum(fall * (6.0 / k), 1)
        # lists are of unlike lengths where rows are ignored: what is past the end has no token
        length = torch.full((rows,), k, device="cuda")
        if case["ignored"]:
            length = 1 + (torch.rand(rows, generator=gen, device="cuda") * k).long().clamp(max=k - 1)
        there = (torch.arange(k, device="cuda") < length[:, None]) & valid[:, None]
        s["index"] = torch.where(there, index, -1).to(torch.int32)
    if case["op"].endswith("train"):
        s["dloss"] = (valid.float() / max(1, sum(is_valid(case)))).contiguous()  # of the mean over the rows that count
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = _linear_inputs(case, gen) if case["op"].startswith("linear") else _head_inputs(case, gen)
    s["case"] = case
    if own:
        s["plan"] = _plan(s)
    return s


# ---------------------------------------------------------------------------- plain forms

def _act(z, kind):
    """The activation and its derivative."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0.0), (z > 0).to(z.dtype)
    if kind == "silu":
        g = 1.0 / (1.0 + torch.exp(-z))
        return z * g, g * (1.0 + z * (1.0 - g))
    if kind == "gelu":
        c = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * c, c + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    a, b = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(a * (z + b * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3.0 * b * z * z)


def _linear(s):
    case, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    if case["bias"]:
        z = z + s["b"].float()
    y, slope = _act(z, case["act"])
    if case["residual"]:
        y = y + s["r"].float()
    if case["op"] == "linear_forward":
        return {"y": y.to(dt)}
    dz = s["dy"].float() * slope
    out = {"y": y.to(dt), "dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt)}
    if case["act"] != "none":
        out["pre"] = z.to(dt)
    if case["bias"]:
        out["db"] = dz.sum(0).to(dt)
    return out


def _loss(s):
    """Cross entropy with one token of weight 1 per row, or with a teacher's probabilities of k tokens."""
    case, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    t = case.get("temperature", 1.0)
    z = (x @ w.t()) * (1.0 / t)
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    if case["op"].startswith("vocab"):
        index, there = s["target"][:, None].clamp(min=0), s["target"][:, None] >= 0
        q = there.float()
        given = torch.zeros_like(lse)
    else:
        index, there = s["index"].long().clamp(min=0), s["index"] >= 0
        u = torch.where(there, s["logit"].float() * (1.0 / t), -math.inf)
        best = u.amax(1, keepdim=True)
        u = torch.where(there, u - best, 0.0)
        q = torch.where(there, torch.exp(u), 0.0)
        norm = q.sum(1, keepdim=True)
        q = torch.where(there, q / norm, 0.0)
        given = torch.where(there, q * (u - torch.log(norm)), 0.0).sum(1)
    valid = there.any(1)
    picked = (q * torch.gather(z, 1, index)).sum(1)
    loss = torch.where(valid, (t * t) * (given + lse - picked), 0.0)
    lse = torch.where(valid, lse, 0.0)
    if case["op"].endswith("forward"):
        return {"loss": loss, "lse": lse}
    p = e / total
    p = p.scatter_add(1, index, -q)
    dz = p * torch.where(valid, s["dloss"] * t, 0.0)[:, None]
    return {"loss": loss, "lse": lse, "dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt)}


# ------------------------------------------------------------------- the framework's calls

def _plan(s):
    """Handles, outputs and workspaces, as a program makes them before its first step."""
    import residual_gradient_compression_gb300 as ac
    case, rows = s["case"], s["case"]["rows"]
    code = ac.BF16 if case["x"] == "bf16" else ac.F32
    p = {"ac": ac}

    def workspace(nbytes):
        return torch.zeros(max(16, nbytes), dtype=torch.uint8, device="cuda")

    if case["op"].startswith("linear"):
        act = {"none": ac.ACT_NONE, "relu": ac.ACT_RELU, "gelu": ac.ACT_GELU, "gelu_tanh": ac.ACT_GELU_TANH,
               "silu": ac.ACT_SILU}[case["act"]]
        p["h"] = ac.adacomp_linear_init(case["din"], case["dout"], code, act)
        need = ac.adacomp_linear_forward_ws_bytes(p["h"], rows)
        p["y"] = torch.empty(rows, case["dout"], dtype=s["x"].dtype, device="cuda")
        p["pre"] = None
        if case["op"] == "linear_train":
            need = max(need, ac.adacomp_linear_backward_ws_bytes(p["h"], rows))
            if case["act"] != "none":
                p["pre"] = torch.empty_like(p["y"])
            p["dx"], p["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
            p["db"] = torch.empty_like(s["b"]) if case["bias"] else None
        p["ws"] = workspace(need)
        return p
    p["h"] = ac.adacomp_vocab_init(case["dim"], case["vocab"], code)
    p["loss"], p["lse"] = (torch.empty(rows, device="cuda") for _ in range(2))
    distill = case["op"].startswith("distill")
    need = (ac.adacomp_distill_forward_ws_bytes(p["h"], rows, case["k"]) if distill
            else ac.adacomp_vocab_loss_forward_ws_bytes(p["h"], rows))
    if case["op"].endswith("train"):
        need = max(need, ac.adacomp_distill_backward_ws_bytes(p["h"], rows, case["k"]) if distill
                   else ac.adacomp_vocab_loss_backward_ws_bytes(p["h"], rows))
        p["dx"], p["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
    p["ws"] = workspace(need)
    return p


def _own(s):
    p, case = s["plan"], s["case"]
    ac, h, op = p["ac"], p["h"], s["case"]["op"]
    if op.startswith("linear"):
        ac.adacomp_linear_forward(h, s["x"], s["w"], p["y"], p["ws"], bias=s["b"], residual=s["r"], pre=p["pre"])
        if op == "linear_forward":
            return {"y": p["y"]}
        ac.adacomp_linear_backward(h, s["dy"], s["x"], s["w"], p["ws"], pre=p["pre"], dx=p["dx"], dw=p["dw"], db=p["db"])
        return {k: p[k] for k in ("y", "dx", "dw", "pre", "db") if p[k] is not None}
    if op.startswith("vocab"):
        ac.adacomp_vocab_loss_forward(h, s["x"], s["w"], s["target"], p["loss"], p["lse"], p["ws"])
        if op.endswith("forward"):
            return {"loss": p["loss"], "lse": p["lse"]}
        ac.adacomp_vocab_loss_backward(h, s["x"], s["w"], s["target"], p["lse"], s["dloss"], p["ws"], dx=p["dx"],
                                       dw=p["dw"])
    else:
        t = case["temperature"]
        ac.adacomp_distill_forward(h, s["x"], s["w"], s["index"], s["logit"], t, p["loss"], p["lse"], p["ws"])
        if op.endswith("forward"):
            return {"loss": p["loss"], "lse": p["lse"]}
        ac.adacomp_distill_backward(h, s["x"], s["w"], s["index"], s["logit"], t, p["lse"], s["dloss"], p["ws"],
                                    dx=p["dx"], dw=p["dw"])
    return {k: p[k] for k in ("loss", "lse", "dx", "dw")}


def run(state):
    if own:
        return _own(state)
    return _linear(state) if state["case"]["op"].startswith("linear") else _loss(state)


# --------------------------------------------------------------------------- in 64 bits

def _exact_linear(s):
    """A block of rows at a time, the sums of the gradients carried along."""
    case, w = s["case"], s["w"].double()
    kind, parts, dw, db = case["act"], [], torch.zeros_like(w), torch.zeros_like(w[:, 0])
    for r in range(0, case["rows"], 4096):
        x = s["x"][r:r + 4096].double()
        pre = torch.einsum("ri,oi->ro", x, w)
        if case["bias"]:
            pre += s["b"].double()[None, :]
        pre.requires_grad_(case["op"] == "linear_train")
        if kind == "relu":
            y = torch.where(pre > 0, pre, torch.zeros_like(pre))
        elif kind == "silu":
            y = pre / (1 + torch.exp(-pre))
        elif kind == "gelu":
            y = pre * torch.special.erfc(-pre / math.sqrt(2)) / 2
        elif kind == "gelu_tanh":  # (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
            y = pre / (1 + torch.exp(-math.sqrt(8 / math.pi) * (pre + 0.044715 * pre ** 3)))
        else:
            y = pre * 1
        part = {}
        if case["op"] == "linear_train":
            dz, = torch.autograd.grad(y, pre, s["dy"][r:r + 4096].double())
            part["dx"] = dz @ w
            dw += torch.einsum("ro,ri->oi", dz, x)
            db += dz.sum(0)
        part["pre"] = pre.detach()
        part["y"] = y.detach() + (s["r"][r:r + 4096].double() if case["residual"] else 0)
        parts.append(part)
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["op"] == "linear_forward":
        return {"y": out["y"]}
    out["dw"] = dw
    if case["bias"]:
        out["db"] = db
    if kind == "none":
        del out["pre"]
    return out


def _exact_loss(s):
    """Only the rows that have a loss, a block of them at a time."""
    case, w = s["case"], s["w"].double()
    rows, dim, t = case["rows"], case["dim"], case.get("temperature", 1.0)
    train = case["op"].endswith("train")
    loss, lse = (torch.zeros(rows, dtype=torch.float64, device=w.device) for _ in range(2))
    dx, dw = torch.zeros(rows, dim, dtype=torch.float64, device=w.device), torch.zeros_like(w)
    index = s["target"][:, None] if case["op"].startswith("vocab") else s["index"].long()
    some = torch.nonzero((index >= 0).any(1))[:, 0]
    for at in some.split(2048):
        x, idx = s["x"][at].double(), index[at]
        z = torch.einsum("ri,vi->rv", x, w) / t
        logp = z - torch.logsumexp(z, 1, keepdim=True)
        lse[at] = (z - logp)[:, 0]
        teacher = torch.zeros_like(idx, dtype=torch.float64) if "logit" not in s else s["logit"][at].double() / t
        logq = torch.log_softmax(teacher.masked_fill(idx < 0, -math.inf), 1)
        q = torch.exp(logq)
        gap = logq - torch.gather(logp, 1, idx.clamp(min=0))
        loss[at] = t * t * torch.where(idx >= 0, q * gap, torch.zeros_like(q)).sum(1)
        if train:
            # d(t^2 KL)/dz: t times the difference of the two distributions
            g = torch.exp(logp)
            g.scatter_add_(1, idx.clamp(min=0), torch.where(idx >= 0, -q, torch.zeros_like(q)))
            g *= t * s["dloss"][at].double()[:, None]
            dx[at] = g @ w
            dw += torch.einsum("rv,ri->vi", g, x)
    out = {"loss": loss, "lse": lse}
    if train:
        out.update(dx=dx, dw=dw)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_linear(s) if case["op"].startswith("linear") else _exact_loss(s)
