"""Plain 64-bit forms of the training operators and the error bounds that their 32-bit
kernels are held to (test helper only).

The bounds are worst-case rounding bounds of any evaluation in fp32 whose sums add at most
`depth` terms in sequence; U is fp32's unit roundoff, and OUT the output type's."""
import torch

U = 2.0 ** -24
OUT = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16)}
#: gate(): exp to 2 + 1.173 |z| ulp, a quotient to 2 ulp, an addition: as CUDA documents them
GATE_ULP, GATE_PER_Z = 6.0, 1.2


def assert_within(got, ref, bound, what):
    """Every element of `got` within `bound` of `ref`; non-finite values in the same places.
    The bounds are relative to normal numbers: a result below them is rounded to half of the
    type's smallest number, after some fp32 products that were rounded so."""
    kind = torch.finfo(got.dtype)
    bound = bound + kind.smallest_normal * kind.eps / 2 + 16 * 2.0 ** -149
    got, ref = got.double(), ref.double()
    fine = torch.isfinite(ref)
    assert torch.equal(fine, torch.isfinite(got)), f"{what}: non-finite values elsewhere"
    over = ((got - ref).abs() - bound)[fine]
    if over.numel() and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError(f"{what}: off by {float((got - ref)[fine].abs().flatten()[i]):.3g}, bound "
                             f"{float(bound.expand_as(ref)[fine].flatten()[i]):.3g}, at {i} of {over.numel()}")


# ------------------------------------------------------------------------------ layer norm

def norm_forward(x, w, b, eps):
    """(y, mean, rstd) and their bounds, in 64 bits."""
    dt = x.dtype
    x, w = x.double(), w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    n = x.shape[1]
    depth = -(-n // 32) + 10
    mean = x.mean(1, keepdim=True)
    dev = x - mean
    var = (dev * dev).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    y = dev * rstd * w + b
    size = x.abs().mean(1, keepdim=True)
    e_mean = depth * U * size
    e_dev = e_mean + U * (x.abs() + mean.abs())  # of x - mean
    # var: its terms' errors (first and second order), and the sum's
    e_var = (2 * dev.abs() * e_dev + e_dev * e_dev).mean(1, keepdim=True) + (depth + 3) * U * var
    # the root's change over that range, bounded by its slope at the lower end
    low = (var + eps - e_var).clamp(min=torch.finfo(torch.float64).tiny)
    e_rstd = torch.where(e_var < var + eps, 1 / torch.sqrt(low) - rstd, torch.inf) + 4 * U * rstd
    e_y = w.abs() * (e_dev * (rstd + e_rstd) + dev.abs() * e_rstd) + 4 * U * (y.abs() + b.abs())
    return (y, mean[:, 0], rstd[:, 0]), (e_y + OUT[dt] * (y.abs() + e_y), e_mean[:, 0], e_rstd[:, 0])


def norm_backward(dy, x, w, mean, rstd, wt):
    """(dx, dw, db) and their bounds, in 64 bits, from the given mean and rstd."""
    dt, rows, n = x.dtype, x.shape[0], x.shape[1]
    depth = -(-n // 32) + 10
    dy, x, w = dy.double(), x.double(), w.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * rstd
    e_xh = rstd * U * (x.abs() + mean.abs()) + 3 * U * xh.abs()
    g = dy * w
    s0, s1 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - s0 - xh * s1)
    e_s0 = (depth + 2) * U * g.abs().mean(1, keepdim=True)
    e_s1 = (depth + 4) * U * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * e_xh).mean(1, keepdim=True)
    e_dx = rstd * (6 * U * (g.abs() + s0.abs() + (xh * s1).abs()) + e_s0 + xh.abs() * e_s1 + e_xh * s1.abs()
                   + e_xh * e_s1)
    dw, db = (dy * xh).sum(0), dy.sum(0)
    e_dw = (rows + 10) * U * (dy * xh).abs().sum(0) + (dy.abs() * e_xh).sum(0)
    e_db = (rows + 10) * U * dy.abs().sum(0)
    return ((dx, dw, db), (e_dx + OUT[dt] * (dx.abs() + e_dx), e_dw + OUT[wt] * (dw.abs() + e_dw),
                           e_db + OUT[wt] * (db.abs() + e_db)))


# ------------------------------------------------------------------------------ recurrence

def _live(lengths, batch, steps, device):
    if lengths is None:
        return torch.ones(batch, steps, 1, dtype=torch.bool, device=device)
    return (torch.arange(steps, device=device)[None, :] < lengths.clamp(0, steps)[:, None])[..., None]


def recurrence(z, x, h0, lengths=None, dy=None, dh_last=None):
    """(y, h_last) or, with dy, (y, h_last, dz, dx, dh0), and their bounds, step by step in
    64 bits. The bound on the state follows the recurrence itself; it is doubled because a
    kernel may form a state from the product of several gates and a state before them."""
    dt = z.dtype
    batch, steps, ch = z.shape
    live = _live(lengths, batch, steps, z.device)
    z = torch.where(live, z.double(), 0.0)
    x = torch.where(live, x.double(), 0.0)
    a, b = torch.sigmoid(z), torch.sigmoid(-z)
    rel = (GATE_ULP + GATE_PER_Z * z.abs()) * 2 * U  # of a and of 1 - a
    h = torch.zeros(batch, ch, dtype=torch.float64, device=z.device) if h0 is None else h0.double()
    err = torch.zeros_like(h)
    before, e_before, hs, e_hs = [], [], [], []
    for t in range(steps):
        before.append(h)
        e_before.append(err)
        new = a[:, t] * h + b[:, t] * x[:, t]
        e = a[:, t] * err + rel[:, t] * (a[:, t] * h.abs() + b[:, t] * x[:, t].abs()) \
            + 4 * U * (a[:, t] * h.abs() + b[:, t] * x[:, t].abs() + new.abs())
        h, err = torch.where(live[:, t], new, h), torch.where(live[:, t], e, err)
        hs.append(torch.where(live[:, t], h, 0.0))
        e_hs.append(torch.where(live[:, t], err, 0.0))
    empty = z
    stack = lambda v: torch.stack(v, 1) if v else empty  # noqa: E731
    y, e_y = stack(hs), 2 * stack(e_hs)
    out = [y, h]
    bound = [e_y + OUT[dt] * (y.abs() + e_y), 2 * err + 2 * U * h.abs()]
    if dy is None:
        return out, bound
    dy = torch.where(live, dy.double(), 0.0)
    g = torch.zeros_like(h) if dh_last is None else dh_last.double()  # reaches h_t from the steps after it
    err = torch.zeros_like(g)
    dzs, dxs, e_dzs, e_dxs = [], [], [], []
    for t in range(steps - 1, -1, -1):
        on = live[:, t]
        full = g + dy[:, t]
        e_full = err + 2 * U * (g.abs() + dy[:, t].abs() + full.abs())
        dx = b[:, t] * full
        diff = before[t] - x[:, t]
        dz = a[:, t] * dx * diff
        e2 = 2 * e_full
        e_dx = b[:, t] * e2 + (rel[:, t] + 3 * U) * dx.abs()
        e_diff = 2 * e_before[t] + 2 * U * (before[t].abs() + x[:, t].abs())
        e_dz = a[:, t] * (b[:, t] * (e2 * diff.abs() + (full.abs() + e2) * e_diff)) + (2 * rel[:, t] + 6 * U) * dz.abs()
        dzs.append(torch.where(on, dz, 0.0))
        dxs.append(torch.where(on, dx, 0.0))
        e_dzs.append(torch.where(on, e_dz, 0.0))
        e_dxs.append(torch.where(on, e_dx, 0.0))
        g, err = (torch.where(on, a[:, t] * full, g),
                  torch.where(on, a[:, t] * e_full + (rel[:, t] + 3 * U) * (a[:, t] * full).abs(), err))
    for v, e in ((dzs, e_dzs), (dxs, e_dxs)):
        v, e = stack(v[::-1]), stack(e[::-1])
        out.append(v)
        bound.append(e + OUT[dt] * (v.abs() + e))
    out.append(g)
    bound.append(2 * err + 2 * U * g.abs())
    return out, bound


# ----------------------------------------------------------------------------------- AdamW

def to_e4m3(v):
    """The nearest e4m3 number (ties to even, largest 448) of fp64 values, by its definition."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def blocks(v, block=256):
    """A flat tensor as rows of `block`, zeros after its end."""
    n = v.numel()
    return torch.nn.functional.pad(v, (0, -n % block)).view(-1, block)
