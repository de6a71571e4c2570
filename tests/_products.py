"""Plain 64-bit forms of the linear layers and of the losses over a vocabulary, and the error bounds that
their kernels are held to (test helper only).

The bounds are worst-case: a product's partial sums are each off by at most 2 U of the terms' magnitudes (U is
fp32's unit roundoff: a partial sum may be truncated), functions by what CUDA documents (exp 2 + 1.173 |x|
units in the last place, erf and tanh 2), and results are rounded once to the output's type."""
import math

import torch

from _train import OUT, U, assert_within  # noqa: F401

PARTS = {torch.float32: 6, torch.bfloat16: 1}  # products of parts that are summed for one of numbers


def slack(terms, dt):
    """Of a sum of products, relative to the sum of their magnitudes."""
    return (PARTS[dt] * terms + 16) * 2 * U + (2.0 ** -22 if dt == torch.float32 else 0.0)


def act(z, kind):
    """The activation and its slope."""
    if kind == "relu":
        return z.clamp(min=0.0), (z > 0).to(z.dtype)
    if kind == "gelu":
        c = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        a, b = math.sqrt(2 / math.pi), 0.044715
        t = torch.tanh(a * (z + b * z ** 3))
        return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t * t) * a * (1 + 3 * b * z * z)
    if kind == "silu":
        g = torch.sigmoid(z)
        return z * g, g * (1 + z * torch.sigmoid(-z))
    return z, torch.ones_like(z)


def linear(x, w, bias, residual, kind):
    """(y, z) and their bounds."""
    dt = x.dtype
    x, w = x.double(), w.double()
    z = x @ w.T
    e = slack(x.shape[1], dt) * (x.abs() @ w.abs().T)
    if bias is not None:
        z = z + bias.double()
        e = e + 2 * U * (z.abs() + bias.double().abs())
    y = act(z, kind)[0]
    # slopes are at most 1.13; a function's own error is 2 units of a value up to |z|, its argument's some more
    e_y = e if kind == "none" else 1.2 * e + 16 * U * z.abs()
    if residual is not None:
        y = y + residual.double()
        e_y = e_y + 2 * U * (y.abs() + residual.double().abs())
    return (y, z), (e_y + OUT[dt] * (y.abs() + e_y), e + OUT[dt] * (z.abs() + e))


def linear_backward(dy, x, w, pre, kind):
    """(dx, dw, db) and their bounds, from the value before the activation as it is given."""
    dt = dy.dtype
    dy, x, w = dy.double(), x.double(), w.double()
    dz = dy if kind == "none" else dy * act(pre.double(), kind)[1]
    # a slope is made of terms up to 3, of functions that are off by a few units each, at worst by 9 times tanh's 10
    e_z = torch.zeros_like(dz) if kind == "none" else dy.abs() * 128 * U + 2 * U * dz.abs()
    e_r = e_z + (OUT[dt] * (dz.abs() + e_z) if dt == torch.bfloat16 and kind != "none" else 0)
    size = dz.abs() + e_r
    out, bound = [], []
    for value, e in ((dz @ w, e_r @ w.abs() + slack(dz.shape[1], dt) * (size @ w.abs())),
                     (dz.T @ x, e_r.T @ x.abs() + slack(dz.shape[0], dt) * (size.T @ x.abs())),
                     (dz.sum(0), e_z.sum(0) + (dz.shape[0] + 10) * U * size.sum(0))):
        out.append(value)
        bound.append(e + OUT[dt] * (value.abs() + e))
    return out, bound


def lists(index, logit, temperature, vocab):
    """(index, q, given, valid): the listed tokens' weights, sum of q log q, and which rows have a loss; and
    the weights' relative error."""
    there = index >= 0
    valid = there.any(1)
    if logit is None:
        return index.clamp(min=0), there.double(), torch.zeros(index.shape[0], device=index.device).double(), valid, 0.0
    u = logit.double() / temperature
    u = torch.where(there, u, -math.inf)
    top = torch.where(valid, u.amax(1), 0.0)[:, None]
    total = torch.exp(u - top).sum(1, keepdim=True)
    q = torch.where(there, torch.exp(u - top) / torch.where(valid[:, None], total, 1.0), 0.0)
    given = torch.where(q > 0, q * torch.log(torch.where(q > 0, q, 1.0)), 0.0).sum(1)
    spread = torch.where(torch.isfinite(u), (u - top).abs() + 2 * u.abs() + 2 * top.abs(), 0.0).amax()
    return index.clamp(min=0).long(), q, given, valid, float(2 * (4 + 2.4 * spread) * U + (index.shape[1] + 16) * U)


def logits(x, w, temperature):
    dt = x.dtype
    x, w = torch.nan_to_num(x.double()), w.double()  # rows without a loss may hold anything
    z = x @ w.T / temperature
    e = slack(x.shape[1], dt) * (x.abs() @ w.abs().T) / temperature + 4 * U * z.abs()
    return z, e


def loss(x, w, index, logit=None, temperature=1.0):
    """(loss, lse) and their bounds; index [rows, k], with a teacher's logits or one target each."""
    t2 = temperature * temperature
    z, e_z = logits(x, w, temperature)
    index, q, given, valid, e_q = lists(index, logit, temperature, w.shape[0])
    lse = torch.logsumexp(z, 1)
    top = z.amax(1, keepdim=True)
    vocab = w.shape[0]
    # of the sum: additions in a row, a dozen rescalings, the terms' own exps weighted by what they add
    rescale = 12 * (2 + 1.2 * (z - top).abs().amax(1)) * 2 * U
    terms = (torch.softmax(z, 1) * (2 + 1.2 * (z - top).abs()) * 2 * U).sum(1)
    e_lse = e_z.amax(1) + (96 + vocab / 8192) * 2 * U + rescale + terms + 4 * U * (1 + lse.abs() + top[:, 0].abs())
    picked, e_p = torch.gather(z, 1, index), torch.gather(e_z, 1, index)
    mean = (q * torch.where(q > 0, picked, 0.0)).sum(1)
    value = given + lse - mean
    gap = (q * (1 + torch.log(torch.where(q > 0, q, 1.0)).abs() + picked.abs())).sum(1)
    e = e_lse + (q * e_p).sum(1) + e_q * gap + (q.shape[1] + 16) * U * (given.abs() + lse.abs() + gap)
    out = (torch.where(valid, t2 * value, 0.0), torch.where(valid, lse, 0.0))
    return out, (t2 * (e + 4 * U * value.abs()), e_lse)


def loss_backward(x, w, index, lse, dloss, logit=None, temperature=1.0):
    """(dx, dw) and their bounds, from the logarithm lse as it is given."""
    dt = x.dtype
    z, e_z = logits(x, w, temperature)
    index, q, _, valid, e_q = lists(index, logit, temperature, w.shape[0])
    lse = torch.where(valid, lse.double(), 0.0)[:, None]
    d = torch.where(valid[:, None], z - lse, 0.0)
    p = torch.exp(d)
    e_p = p * torch.expm1(e_z + 2 * U * d.abs() + (2 + 1.2 * d.abs()) * 2 * U)
    f = torch.where(valid, dloss.double() * temperature, 0.0)[:, None]
    qs = torch.zeros_like(p).scatter_add_(1, index, q)
    dz = f * (p - qs)
    e = f.abs() * (e_p + (e_q + (q.shape[1] + 2) * U) * qs + 2 * U * (p + qs)) + 4 * U * dz.abs()
    e = e + (OUT[dt] * (dz.abs() + e) if dt == torch.bfloat16 else 0) + 2.0 ** -133
    x = torch.where(valid[:, None], torch.nan_to_num(x.double()), 0.0)
    w, size = w.double(), dz.abs() + e
    # the vocabulary's pieces are added up in fp32
    out, bound = [], []
    for value, b in ((dz @ w, e @ w.abs() + (slack(dz.shape[1], dt) + 64 * U) * (size @ w.abs())),
                     (dz.T @ x, e.T @ x.abs() + slack(dz.shape[0], dt) * (size.T @ x.abs()))):
        out.append(value)
        bound.append(b + OUT[dt] * (value.abs() + b))
    return out, bound


def strided(t, pad, shift=0):
    """A copy of the matrix t with rows `pad` elements further apart, beginning `shift` elements past an
    aligned address; what lies between the rows is NaN."""
    rows, cols = t.shape
    flat = torch.full((rows * (cols + pad) + shift + 16,), math.nan, dtype=t.dtype, device=t.device)
    view = flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view
