"""Losses over a vocabulary (GPU): softmax cross entropy and distillation, forward and backward, against
plain forms in 64 bits, within bounds derived from the operations."""
import math

import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace
from _products import assert_within, loss as loss_ref, loss_backward as backward_ref, strided

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _inputs(rows, dim, vocab, dt, seed=0, sharp=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, dim, generator=g, device="cuda").to(dt)
    w = (torch.randn(vocab, dim, generator=g, device="cuda") * (sharp * dim ** -0.5)).to(dt)
    target = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    return x, w, target, torch.randn(rows, generator=g, device="cuda"), g


def _teacher(rows, k, vocab, g, ragged):
    index = torch.rand(rows, vocab, generator=g, device="cuda").topk(min(k, vocab), 1).indices
    if index.shape[1] < k:
        index = torch.nn.functional.pad(index, (0, k - index.shape[1]), value=-1)
    if ragged:
        length = torch.randint(0, k + 1, (rows, 1), generator=g, device="cuda")
        index = torch.where(torch.arange(k, device="cuda") < length, index, -1)
    return index.to(torch.int32), 3 * torch.randn(rows, k, generator=g, device="cuda")


class Head:
    def __init__(self, dim, vocab, dt):
        self.h = ac.adacomp_vocab_init(dim, vocab, ac.BF16 if dt == BF16 else ac.F32)
        self.dim, self.vocab, self.dt = dim, vocab, dt

    def _ws(self, name, rows, *k):
        return workspace(getattr(ac, f"adacomp_{name}_ws_bytes")(self.h, rows, *k)).fill_(255)

    def forward(self, x, w, target, teacher=None, t=1.0):
        rows = x.shape[0]
        loss, lse = (torch.full((rows,), NAN, device="cuda") for _ in range(2))
        if teacher is None:
            ac.adacomp_vocab_loss_forward(self.h, x, w, target, loss, lse, self._ws("vocab_loss_forward", rows))
        else:
            ac.adacomp_distill_forward(self.h, x, w, *teacher, t, loss, lse,
                                       self._ws("distill_forward", rows, teacher[0].shape[1]))
        return loss, lse

    def backward(self, x, w, target, lse, dloss, teacher=None, t=1.0, dx=None, dw=None):
        rows = x.shape[0]
        dx = torch.full((rows, self.dim), NAN, dtype=self.dt, device="cuda") if dx is None else dx
        dw = torch.full((self.vocab, self.dim), NAN, dtype=self.dt, device="cuda") if dw is None else dw
        if teacher is None:
            ac.adacomp_vocab_loss_backward(self.h, x, w, target, lse, dloss, self._ws("vocab_loss_backward", rows), dx, dw)
        else:
            ac.adacomp_distill_backward(self.h, x, w, *teacher, t, lse, dloss,
                                        self._ws("distill_backward", rows, teacher[0].shape[1]), dx, dw)
        return dx, dw


def _check(x, w, target, dloss, teacher=None, t=1.0, head=None):
    head = head or Head(x.shape[1], w.shape[0], x.dtype)
    index, logit = (target[:, None], None) if teacher is None else (teacher[0], teacher[1].float())
    loss, lse = head.forward(x, w, target, teacher, t)
    ref, bound = loss_ref(x, w, index, logit, t)
    assert_within(loss, ref[0], bound[0], "loss")
    assert_within(lse, ref[1], bound[1], "lse")
    got = head.backward(x, w, target, lse, dloss, teacher, t)
    ref, bound = backward_ref(x, w, index, lse, dloss, logit, t)
    assert_within(got[0], ref[0], bound[0], "dx")
    assert_within(got[1], ref[1], bound[1], "dw")


SIZES = [(1, 1, 1), (1, 64, 1000), (2, 33, 2), (5, 8, 257), (32, 256, 5000), (100, 72, 31), (129, 65, 1025),
         (200, 128, 2304), (257, 40, 4099), (64, 501, 10007), (300, 24, 255), (140, 264, 513)]


@DTYPES
@pytest.mark.parametrize("rows,dim,vocab", SIZES)
def test_cross_entropy(rows, dim, vocab, dt):
    x, w, target, dloss, _ = _inputs(rows, dim, vocab, dt)
    if rows > 4:
        target[::3] = -100
        target[1] = vocab - 1
    _check(x, w, target.to(torch.int32) if rows % 2 else target, dloss)


@DTYPES
@pytest.mark.parametrize("rows,dim,vocab,k,t,ragged", [
    (1, 16, 10, 1, 1.0, False), (3, 64, 300, 20, 2.0, False), (130, 40, 1000, 64, 1.0, True), (40, 72, 70, 100, 0.5, True),
    (200, 128, 2500, 256, 3.0, True), (65, 501, 4099, 33, 1.5, False), (17, 8, 33, 33, 1.0, True)])
def test_distillation(rows, dim, vocab, k, t, ragged, dt):
    x, w, target, dloss, g = _inputs(rows, dim, vocab, dt, 1)
    index, logit = _teacher(rows, k, vocab, g, ragged)
    _check(x, w, target, dloss, (index, logit.to(BF16) if rows % 2 else logit), t)


@DTYPES
def test_more_than_one_piece(dt):
    """So many rows that the backward pass takes the vocabulary in pieces of 2048."""
    x, w, target, dloss, g = _inputs(70_000, 8, 4500, dt, 2)
    target[5::7] = -1
    _check(x[:30], w, target[:30], dloss[:30])
    head = Head(8, 4500, dt)
    loss, lse = head.forward(x, w, target)
    dx, dw = head.backward(x, w, target, lse, dloss)
    ref, bound = [torch.zeros(4500, 8, dtype=torch.float64, device="cuda") for _ in range(2)], None
    total = [0.0, 0.0]
    for at in range(0, 70_000, 10_000):
        part = slice(at, at + 10_000)
        r, b = loss_ref(x[part], w, target[part][:, None])
        assert_within(loss[part], r[0], b[0], "loss")
        r, b = backward_ref(x[part], w, target[part][:, None], lse[part], dloss[part])
        assert_within(dx[part], r[0], b[0], "dx")
        total = [total[0] + r[1], total[1] + b[1]]
    # the bound of a sum of all rows: that of each part's sums, times the parts
    assert_within(dw, total[0], 7 * total[1], "dw")


@DTYPES
def test_sharp_and_flat_distributions(dt):
    """Logits of hundreds, where all but one of the probabilities vanish; and logits that are all alike."""
    x, w, target, dloss, g = _inputs(150, 32, 700, dt, 3, sharp=100.0)
    _check(x, w, target, dloss)
    best = (x.double() @ w.double().T).argmax(1)
    _check(x, w, best, dloss)
    _check(x, w, target, dloss, _teacher(150, 16, 700, g, False), 1.0)
    w = w[:1].expand(700, 32)
    _check(x, w, target, dloss)
    loss, lse = Head(32, 700, dt).forward(torch.zeros_like(x), w, target)
    assert (lse - math.log(700)).abs().max() < 1e-5 and (loss - math.log(700)).abs().max() < 1e-5


@DTYPES
def test_rows_without_a_loss_may_hold_anything(dt):
    x, w, target, dloss, g = _inputs(200, 48, 600, dt, 4)
    none = torch.arange(200, device="cuda") % 3 == 1
    target[none] = torch.tensor([-1, -100, -2 ** 40], device="cuda").repeat(30)[:int(none.sum())]
    x[none] = torch.tensor([NAN, math.inf, -math.inf], dtype=dt, device="cuda").repeat(30)[:int(none.sum())][:, None]
    dloss[none] = NAN
    _check(x, w, target, dloss)
    index, logit = _teacher(200, 12, 600, g, True)
    index[none] = -1
    logit[index < 0] = NAN
    _check(x, w, target, dloss, (index, logit))


@DTYPES
@pytest.mark.parametrize("rows", [1023, 1024, 1025, 2049])
def test_rows_with_a_loss_around_the_sizes_that_one_block_lists(rows, dt):
    """Few of them, none of the first, the last one among them; all of them; and those of lists."""
    x, w, target, dloss, g = _inputs(rows, 24, 300, dt, 21)
    _check(x, w, target, dloss)
    some = torch.full_like(target, -1)
    some[rows // 2 + 3::37] = target[rows // 2 + 3::37]
    some[-1] = target[-1]
    _check(x, w, some.to(torch.int32), dloss)
    index, logit = _teacher(rows, 7, 300, g, True)
    index[:rows // 3] = -1
    _check(x, w, target, dloss, (index, logit))


@DTYPES
def test_no_row_has_a_loss(dt):
    x, w, target, dloss, _ = _inputs(150, 40, 300, dt, 5)
    head = Head(40, 300, dt)
    target.fill_(-1)
    loss, lse = head.forward(x, w, target)
    dx, dw = head.backward(x, w, target, lse, dloss)
    assert not loss.any() and not lse.any() and not dx.any() and not dw.any()
    none = torch.empty(0, 40, dtype=dt, device="cuda")
    head.forward(none, w, target[:0])
    dx, dw = head.backward(none, w, target[:0], lse[:0], dloss[:0])
    assert not dw.any()


@DTYPES
def test_tokens_that_are_not_there_are_not_silent(dt):
    """A target past the vocabulary: that row's loss and dx are NaN, and dw is; the other rows are as without it."""
    x, w, target, dloss, g = _inputs(140, 40, 300, dt, 6)
    head = Head(40, 300, dt)
    loss, lse = head.forward(x, w, target)
    dx, _ = head.backward(x, w, target, lse, dloss)
    for far in (300, 2 ** 40):
        bad = target.clone()
        bad[77] = far
        got, lse_bad = head.forward(x, w, bad)
        assert torch.isnan(got[77]) and torch.equal(lse, lse_bad)
        gx, gw = head.backward(x, w, bad, lse, dloss)
        assert torch.isnan(gx[77]).all() and torch.isnan(gw).all()
        for a, b in ((got, loss), (gx, dx)):
            a[77] = b[77]
            assert torch.equal(a, b)
    index, logit = _teacher(140, 9, 300, g, False)
    index[77, 3] = 300
    logit[78] = -math.inf
    logit[79, 0] = NAN
    loss, lse = head.forward(x, w, None, (index, logit))
    assert torch.equal(torch.isnan(loss).nonzero()[:, 0].cpu(), torch.tensor([77, 78, 79]))
    gx, gw = head.backward(x, w, None, lse, dloss, (index, logit))
    assert torch.isnan(gx[77:80]).all() and torch.isfinite(gx[:77]).all() and torch.isfinite(gx[80:]).all()


@DTYPES
def test_tokens_listed_twice_and_impossible_ones(dt):
    x, w, target, dloss, g = _inputs(131, 40, 300, dt, 7)
    index, logit = _teacher(131, 10, 300, g, False)
    index[:, 5] = index[:, 2]
    index[3] = 17
    logit[::2, 4] = -math.inf
    _check(x, w, target, dloss, (index, logit))


@DTYPES
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (8, 0), (3, 5)])
@pytest.mark.parametrize("rows", [3, 150])
def test_strides_and_alignment(rows, pad, shift, dt):
    dim, vocab = 104, 700
    x, w, target, dloss, g = _inputs(rows, dim, vocab, dt, 8)
    index, logit = _teacher(rows, 11, vocab, g, True)
    place = lambda v: strided(v, pad, shift)  # noqa: E731
    wide = torch.full((rows, 15), -7, dtype=torch.int32, device="cuda")
    wide[:, 2:13] = index
    head = Head(dim, vocab, dt)
    buffers = [place(torch.zeros(n, dim, dtype=dt, device="cuda")) for n in (rows, vocab)]
    teacher = (wide[:, 2:13], place(logit))
    loss, lse = head.forward(place(x), place(w), target, teacher, 2.0)
    ref, bound = loss_ref(x, w, index, logit, 2.0)
    assert_within(loss, ref[0], bound[0], "loss")
    got = head.backward(place(x), place(w), target, lse, dloss, teacher, 2.0, *buffers)
    ref, bound = backward_ref(x, w, index, lse, dloss, logit, 2.0)
    for name, a, r, b in zip(("dx", "dw"), got, ref, bound):
        assert_within(a, r, b, name)
        whole = torch.as_strided(a, (a._base.numel(),), (1,), 0)
        inside = torch.zeros_like(whole, dtype=torch.bool)
        torch.as_strided(inside, a.shape, a.stride(), a.storage_offset()).fill_(True)
        assert torch.isnan(whole[~inside]).all()


@DTYPES
def test_one_value_of_dloss_for_all_rows_and_each_gradient_alone(dt):
    x, w, target, dloss, _ = _inputs(150, 40, 700, dt, 9)
    head = Head(40, 700, dt)
    _, lse = head.forward(x, w, target)
    one = torch.full((1,), 1 / 150, device="cuda")
    dx, dw = head.backward(x, w, target, lse, one)
    wx, ww = head.backward(x, w, target, lse, one.expand(150).contiguous())
    assert torch.equal(dx, wx) and torch.equal(dw, ww)
    ws = workspace(ac.adacomp_vocab_loss_backward_ws_bytes(head.h, 150))
    for name, want in (("dx", dx), ("dw", dw)):
        got = torch.empty_like(want)
        ac.adacomp_vocab_loss_backward(head.h, x, w, target, lse, one, ws, **{name: got})
        assert torch.equal(got, want), name


@DTYPES
@pytest.mark.parametrize("rows", [4, 300])
def test_determinism_streams_and_graphs(rows, dt):
    """The same bits again, on another stream, and from a replayed graph with other targets in place, so that
    another number of rows has a loss."""
    x, w, target, dloss, g = _inputs(rows, 72, 1000, dt, 10)
    target[2::5] = -1
    head = Head(72, 1000, dt)

    def step(target):
        loss, lse = head.forward(x, w, target)
        return (loss, lse, *head.backward(x, w, target, lse, dloss))

    first = step(target)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = step(target)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    ws = workspace(max(ac.adacomp_vocab_loss_forward_ws_bytes(head.h, rows), ac.adacomp_vocab_loss_backward_ws_bytes(head.h, rows)))
    now = torch.full_like(target, -1)
    out = [torch.empty_like(t) for t in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ac.adacomp_vocab_loss_forward(head.h, x, w, now, out[0], out[1], ws)
        ac.adacomp_vocab_loss_backward(head.h, x, w, now, out[1], dloss, ws, out[2], out[3])
    graph.replay()
    assert not out[0].any() and not out[3].any()
    for _ in range(2):
        now.copy_(target)
        graph.replay()
        for a, b in zip(first, out):
            assert torch.equal(a, b)


@pytest.mark.parametrize("teach", [False, True])
def test_gradients_against_differences(teach):
    """In fp32: the loss's change along a direction, from central differences in 64 bits (their h^2 term is below
    1e-7 of the directions' size)."""
    x, w, target, dloss, g = _inputs(20, 24, 50, F32, 11)
    teacher, t = (_teacher(20, 6, 50, g, False), 2.0) if teach else (None, 1.0)
    head = Head(24, 50, F32)
    _, lse = head.forward(x, w, target, teacher, t)
    grads = head.backward(x, w, target, lse, dloss, teacher, t)
    for gradient, value in zip(grads, (x, w)):
        way = torch.randn(value.shape, generator=g, device="cuda", dtype=torch.float64)

        def total(s):
            at = [v.double() + s * way if v is value else v.double() for v in (x, w)]
            logp = torch.log_softmax(at[0] @ at[1].T / t, 1)
            if teacher is None:
                each = -logp.gather(1, target[:, None])[:, 0]
            else:
                logq = torch.log_softmax(teacher[1].double() / t, 1)
                each = t * t * (torch.exp(logq) * (logq - logp.gather(1, teacher[0].long()))).sum(1)
            return (dloss.double() * each).sum()

        slope = (total(1e-4) - total(-1e-4)) / 2e-4
        assert abs(slope - (gradient.double() * way).sum()) < 1e-5 * (gradient.double().abs() * way.abs()).sum() + 1e-5
