"""Products whose results are whole numbers below 2^24, so that nothing may be rounded or lost (GPU): every term counts, fp32
operands need all three of their parts, and bf16 results are the exact sums rounded once. On each way that a product takes:
few rows, small matrices, tiles of the tensor cores, sums in parts, both gradients at once, a vocabulary in pieces."""
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _signs(rows, cols, g):
    return torch.randint(0, 2, (rows, cols), generator=g, device="cuda").float() * 2 - 1


def _with_large(t, dt, g):
    """In one place of each row or column, whichever are fewer, and never two in a line, a number with as many bits as the
    type has (fp32 23, so that what is added stays below 2^24); the last row's and column's are among them."""
    n = min(t.shape)
    rows = t.shape[0] - 1 - torch.randperm(t.shape[0], generator=g, device="cuda")[:n]
    cols = torch.randperm(t.shape[1], generator=g, device="cuda")[:n]
    rows[0], cols[0] = t.shape[0] - 1, t.shape[1] - 1
    keep = ((rows != t.shape[0] - 1) & (cols != t.shape[1] - 1)) | (torch.arange(n, device="cuda") == 0)
    bits = 23 if dt == F32 else 8
    large = torch.randint(2 ** (bits - 1), 2 ** bits, (n,), generator=g, device="cuda") | 1
    t = t.clone()
    t[rows[keep], cols[keep]] = large[keep].float()
    return t


def _same(got, ref, what, size=None, terms=0):
    """Exactly; or, where bf16 values are taken in two parts, of which the second is 2^-24 of a value that needs none (so that
    an infinite factor meets no 0): off by that of the terms' magnitudes `size`, by a truncation of as much in each of the
    steps of 16 terms of both parts, and rounded once."""
    assert ref.abs().max() < 2 ** 24
    if size is None:
        assert torch.equal(got, ref.float().to(got.dtype)), what
        return
    off = size * (2.0 ** -24 + 2 * -(-terms // 16) * 2.0 ** -23)
    over = (got.double() - ref).abs() - 2.0 ** -8 * ref.abs() - off * (1 + 2.0 ** -8)
    assert float(over.max()) <= 0, what


SIZES = [(1, 8200, 48), (1, 8203, 50), (5, 5001, 70), (8, 520, 5000), (16, 4104, 33), (9, 130, 40), (17, 5000, 1000), (40, 1000, 60),
         (60, 2000, 31), (64, 800, 500), (70, 6000, 200), (257, 700, 300), (300, 4096, 129), (300, 4097, 1001), (2500, 1000, 1500),
         (2048, 1024, 1024), (1300, 96, 1100), (3001, 1001, 777), (20000, 72, 136), (100, 3000, 3000)]


@DTYPES
@pytest.mark.parametrize("large", ["x", "w", "dy"])
@pytest.mark.parametrize("rows,din,dout", SIZES)
def test_linear(rows, din, dout, large, dt):
    g = torch.Generator(device="cuda").manual_seed(rows + din)
    t = {"x": _signs(rows, din, g), "w": _signs(dout, din, g), "dy": _signs(rows, dout, g)}
    t[large] = _with_large(t[large], dt, g)
    t = {k: v.to(dt) for k, v in t.items()}
    x, w, dy = (t[k].double() for k in ("x", "w", "dy"))
    h = ac.adacomp_linear_init(din, dout, ac.BF16 if dt == BF16 else ac.F32)
    y, dx, dw = (torch.full_like(t[k], NAN) for k in ("dy", "x", "w"))
    ac.adacomp_linear_forward(h, t["x"], t["w"], y, workspace(ac.adacomp_linear_forward_ws_bytes(h, rows)).fill_(255))
    _same(y, x @ w.T, "y")
    ws = workspace(ac.adacomp_linear_backward_ws_bytes(h, rows)).fill_(255)
    ac.adacomp_linear_backward(h, t["dy"], t["x"], t["w"], ws, dx=dx, dw=dw)
    _same(dx, dy @ w, "dx")
    _same(dw, dy.T @ x, "dw")


@pytest.mark.parametrize("rows,din,dout", SIZES)
def test_middle_parts_of_both(rows, din, dout):
    """fp32: numbers of 12 bits, two parts each, times such numbers: one term, the last, is not 0."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, w = torch.zeros(rows, din, device="cuda"), torch.zeros(dout, din, device="cuda")
    x[:, -1], w[:, -1] = ((torch.randint(2 ** 11, 2 ** 12, (n,), generator=g, device="cuda") | 1).float() for n in (rows, dout))
    h = ac.adacomp_linear_init(din, dout)
    y = torch.full((rows, dout), NAN, device="cuda")
    ac.adacomp_linear_forward(h, x, w, y, workspace(ac.adacomp_linear_forward_ws_bytes(h, rows)).fill_(255))
    _same(y, x.double() @ w.double().T, "y")


# dims are odd and even; a vocabulary in pieces of 2048 tokens; few rows against many tokens; sums in parts
HEADS = [(1, 2056, 20000), (20, 200, 5001), (40, 8, 65536), (300, 72, 1300), (512, 64, 20001), (2003, 501, 10007), (9000, 200, 300),
         (70_000, 8, 4500), (70_001, 9, 4300)]


def _head(rows, dim, vocab, dt, g):
    """Hidden states and weights without a column in common, so that all logits are 0 and, from an lse of 0, all
    probabilities 1: dx is dloss times the sum of the weights but for the token's, dw the sum of the rows' but the token's."""
    half = dim // 2
    x, w = _signs(rows, dim, g), _signs(vocab, dim, g)
    x[:, half:], w[:, :half] = 0, 0
    w[:, half:] = _with_large(w[:, half:], dt, g)
    return x, w, half


@DTYPES
@pytest.mark.parametrize("large", ["dloss", "x"])
@pytest.mark.parametrize("rows,dim,vocab", HEADS)
def test_cross_entropys_gradients(rows, dim, vocab, large, dt):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, w, half = _head(rows, dim, vocab, dt, g)
    target = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    target[torch.arange(rows, device="cuda") % 5 == 3] = -1
    for i, t in enumerate((vocab - 1, 2047, 2048, 4095, 4096)):
        if t < vocab and i < rows:
            target[i] = t
    dloss = _signs(rows, 1, g)[:, 0]
    if large == "x":
        x[:, :half] = _with_large(x[:, :half], dt, g)
    else:  # one row's gradient needs all parts; its dx is too large to be exact
        w[:, half:] = w[:, half:].sign()
        at = rows - 1 if int(target[-1]) >= 0 else 0
        dloss[at] = 2 ** 22 + 2 ** 11 + 1 if dt == F32 else 131.0
    x, w = x.to(dt), w.to(dt)
    h = ac.adacomp_vocab_init(dim, vocab, ac.BF16 if dt == BF16 else ac.F32)
    dx, dw = torch.full_like(x, NAN), torch.full_like(w, NAN)
    ws = workspace(ac.adacomp_vocab_loss_backward_ws_bytes(h, rows)).fill_(255)
    ac.adacomp_vocab_loss_backward(h, x, w, target, torch.zeros(rows, device="cuda"), dloss, ws, dx=dx, dw=dw)
    f = torch.where(target >= 0, dloss.double(), 0.0)
    at, xd, wd = target.clamp(min=0), x.double(), w.double()
    want_x = f[:, None] * (wd.sum(0) - wd[at])
    want_w = (f @ xd).expand(vocab, dim).clone().index_add_(0, at, -f[:, None] * xd)
    two = dt == BF16 and rows <= 32
    if large == "x":
        _same(dx, want_x, "dx", f.abs()[:, None] * wd.abs().sum(0) if two else None, vocab)
    _same(dw, want_w, "dw", f.abs() @ xd.abs() if two else None, rows)


@DTYPES
@pytest.mark.parametrize("rows,dim,vocab", HEADS)
def test_distillations_gradients(rows, dim, vocab, dt):
    """Eight listed tokens of equal logits, on both sides of each piece's end: a quarter of the gradient is each token's at a
    temperature of 2, and twice that of one that is listed twice."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, w, half = _head(rows, dim, vocab, dt, g)
    w[:, half:] = w[:, half:].sign() * 4
    x *= 4
    index = torch.randint(0, vocab, (rows, 8), generator=g, device="cuda")
    ends = [t for t in (0, 127, 128, 2047, 2048, 4095, 4096, vocab - 1) if t < vocab]
    index[::2, :len(ends)] = torch.tensor(ends, device="cuda")
    index[1::6, 3] = index[1::6, 1]
    index[2::7] = -1
    dloss = _signs(rows, 1, g)[:, 0]
    x, w = x.to(dt), w.to(dt)
    h = ac.adacomp_vocab_init(dim, vocab, ac.BF16 if dt == BF16 else ac.F32)
    dx, dw = torch.full_like(x, NAN), torch.full_like(w, NAN)
    ws = workspace(ac.adacomp_distill_backward_ws_bytes(h, rows, 8)).fill_(255)
    logit = torch.full((rows, 8), 0.5, device="cuda")
    ac.adacomp_distill_backward(h, x, w, index.to(torch.int32), logit, 2.0, torch.zeros(rows, device="cuda"), dloss, ws, dx=dx, dw=dw)
    f = torch.where(index[:, 0] >= 0, 2 * dloss.double(), 0.0)
    at, xd, wd = index.clamp(min=0), x.double(), w.double()
    want_x, want_w = wd.sum(0).expand(rows, dim).clone(), (f @ xd).expand(vocab, dim).clone()
    for i in range(8):
        want_x -= wd[at[:, i]] / 8
        want_w.index_add_(0, at[:, i], -f[:, None] * xd / 8)
    two = dt == BF16 and rows <= 32
    _same(dx, f[:, None] * want_x, "dx", f.abs()[:, None] * wd.abs().sum(0) if two else None, vocab)
    _same(dw, want_w, "dw", f.abs() @ xd.abs() if two else None, rows)


@DTYPES
@pytest.mark.parametrize("rows,dim,vocab", [(1, 64, 300), (33, 300, 5000), (300, 73, 2100), (1500, 96, 30011)])
def test_losses_of_whole_numbers(rows, dim, vocab, dt):
    """One token's logit is so far above the others' that it is lse itself, and the loss a difference of two logits. Each
    row selects a column of the weights, whose numbers have all of the type's bits."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, w = torch.zeros(rows, dim, device="cuda"), torch.zeros(vocab, dim, device="cuda")
    column = torch.randint(0, dim, (rows,), generator=g, device="cuda")
    column[-1] = dim - 1
    x[torch.arange(rows, device="cuda"), column] = 1
    bits = 23 if dt == F32 else 8
    w[:] = torch.randint(1, 2 ** (bits - 1), (vocab, dim), generator=g, device="cuda").float()
    if dt == BF16:
        w *= 4  # of 4, so that a token apart from the others is more than 104 apart
    top = torch.randint(0, vocab, (dim,), generator=g, device="cuda")
    top[-1] = vocab - 1
    w[top, torch.arange(dim, device="cuda")] = 2.0 ** 23 + 1 if dt == F32 else 1016.0
    x, w = x.to(dt), w.to(dt)
    target = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    h = ac.adacomp_vocab_init(dim, vocab, ac.BF16 if dt == BF16 else ac.F32)
    loss, lse = (torch.full((rows,), NAN, device="cuda") for _ in range(2))
    ac.adacomp_vocab_loss_forward(h, x, w, target, loss, lse, workspace(ac.adacomp_vocab_loss_forward_ws_bytes(h, rows)).fill_(255))
    z = w.double()[:, column].T
    _same(lse, z.amax(1), "lse")
    _same(loss, z.amax(1) - z.gather(1, target[:, None])[:, 0], "loss")
