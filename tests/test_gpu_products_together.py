"""Linear layers and losses over a vocabulary as they are used together (GPU): the example model's gradients against
torch's in 64 bits and against differences, a distilled student's, and calls from several threads and streams."""
import os
import sys
import threading

import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _plain_loss(weights, tokens, blocks, eps=1e-5):
    """The example's model and loss, step by step in the weights' type."""
    def norm(x, w, b):
        return (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, unbiased=False, keepdim=True) + eps) * w + b

    x = weights[0][tokens[:, :-1]]
    for i in range(blocks):
        nw, nb, gates, out = weights[1 + 4 * i:5 + 4 * i]
        z, u = (norm(x, nw, nb) @ gates.T).chunk(2, -1)
        h, hs = torch.zeros_like(u[:, 0]), []
        for t in range(z.shape[1]):
            a = torch.sigmoid(z[:, t])
            h = a * h + (1 - a) * u[:, t]
            hs.append(h)
        x = x + torch.stack(hs, 1) @ out.T
    logits = norm(x, weights[-2], weights[-1]) @ weights[0].T
    target = tokens[:, 1:].reshape(-1, 1)
    return -torch.log_softmax(logits.reshape(target.shape[0], -1), 1).gather(1, target).mean()


@pytest.mark.parametrize("rows,length", [(3, 9), (16, 40)])
def test_the_examples_gradients(rows, length):
    """fp32 through some ten operators: a relative error of 2^-24 each, amplified by sums of up to 640 rows, whose
    magnitudes exceed their results some tens of times, stays below 2^-24 * 10 * 640 = 4e-4 of a gradient's largest
    value, by a wide margin of what the signs leave."""
    import recurrent_lm
    model = recurrent_lm.Model(seed=4)
    for w in model.weights[:1]:
        with torch.no_grad():
            w.mul_(30.0)  # logits that differ
    tokens = recurrent_lm.Text().batch(rows, length)
    loss = model.loss(tokens)
    grads = torch.autograd.grad(loss, model.weights)
    wide = [w.detach().double().requires_grad_() for w in model.weights]
    ref = _plain_loss(wide, tokens, model.blocks)
    refs = torch.autograd.grad(ref, wide)
    assert abs(float(loss.detach()) - float(ref.detach())) < 1e-5 * float(ref.detach())
    for i, (a, b) in enumerate(zip(grads, refs)):
        assert (a.double() - b).abs().max() <= 4e-4 * b.abs().max(), i
    g = torch.Generator(device="cuda").manual_seed(5)
    way = [torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64) for w in wide]
    with torch.no_grad():
        total = [_plain_loss([w + s * 1e-5 * d for w, d in zip(wide, way)], tokens, model.blocks) for s in (1, -1)]
    slope = float(total[0] - total[1]) / 2e-5
    want = float(sum((a.double() * d).sum() for a, d in zip(grads, way)))
    size = float(sum((a.double() * d).abs().sum() for a, d in zip(grads, way)))
    assert abs(slope - want) < 1e-4 * size


def test_a_distilled_students_gradients():
    """A layer with activation and residual under a teacher's loss, in fp32: the gradients of both weights against torch's
    in 64 bits, and within the same reasoning as above of sums of 150 rows or 600 tokens: 2^-24 * 6 operators * 600 = 2e-4."""
    g = torch.Generator(device="cuda").manual_seed(6)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows, width, vocab, k, t = 150, 64, 600, 12, 2.0
    x, w1, w2 = n(rows, width), n(width, width) * 0.125, n(vocab, width) * 0.125
    index = torch.rand(rows, vocab, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    logit = 3 * n(rows, k)
    layer, head = ac.adacomp_linear_init(width, width, ac.F32, ac.ACT_GELU), ac.adacomp_vocab_init(width, vocab)
    ws = workspace(max(ac.adacomp_linear_backward_ws_bytes(layer, rows), ac.adacomp_linear_forward_ws_bytes(layer, rows),
                       ac.adacomp_distill_forward_ws_bytes(head, rows, k), ac.adacomp_distill_backward_ws_bytes(head, rows, k)))
    loss, lse, mean = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.full((1,), 1 / rows, device="cuda")
    y, pre, dy, dw1, dw2 = (torch.empty_like(v) for v in (x, x, x, w1, w2))
    ac.adacomp_linear_forward(layer, x, w1, y, ws, residual=x, pre=pre)
    ac.adacomp_distill_forward(head, y, w2, index, logit, t, loss, lse, ws)
    ac.adacomp_distill_backward(head, y, w2, index, logit, t, lse, mean, ws, dx=dy, dw=dw2)
    ac.adacomp_linear_backward(layer, dy, x, w1, ws, pre=pre, dw=dw1)
    a, b = w1.double().requires_grad_(), w2.double().requires_grad_()
    hidden = torch.nn.functional.gelu(x.double() @ a.T) + x.double()
    logp = torch.log_softmax(hidden @ b.T / t, 1).gather(1, index.long())
    logq = torch.log_softmax(logit.double() / t, 1)
    ref = t * t * (torch.exp(logq) * (logq - logp)).sum(1)
    assert (loss - ref).abs().max() < 2e-4 * ref.abs().max()
    for got, want in zip((dw1, dw2), torch.autograd.grad(ref.mean(), (a, b))):
        assert (got - want).abs().max() < 2e-4 * want.abs().max()


def test_threads_and_streams_with_workspaces_of_their_own():
    """Four host threads, each on its own stream with its own workspace and one handle for all: the results of one
    after the other."""
    g = torch.Generator(device="cuda").manual_seed(7)
    sizes = [(5, 300), (130, 300), (700, 300), (64, 300)]
    h = ac.adacomp_linear_init(300, 520, ac.BF16, ac.ACT_SILU)
    v = ac.adacomp_vocab_init(300, 1500, ac.BF16)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    w, head = n(520, 300) * 0.06, n(1500, 300) * 0.1
    xs = [n(*s) for s in sizes]
    targets = [torch.randint(0, 1500, (s[0],), generator=g, device="cuda") for s in sizes]

    def run(i):
        rows = sizes[i][0]
        y = torch.empty(rows, 520, dtype=torch.bfloat16, device="cuda")
        loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        dx, dw = torch.empty_like(xs[i]), torch.empty_like(head)
        ws = workspace(max(ac.adacomp_linear_forward_ws_bytes(h, rows), ac.adacomp_vocab_loss_backward_ws_bytes(v, rows),
                           ac.adacomp_vocab_loss_forward_ws_bytes(v, rows)))
        for _ in range(10):
            ac.adacomp_linear_forward(h, xs[i], w, y, ws)
            ac.adacomp_vocab_loss_forward(v, xs[i], head, targets[i], loss, lse, ws)
            ac.adacomp_vocab_loss_backward(v, xs[i], head, targets[i], lse, loss, ws, dx=dx, dw=dw)
        return y, loss, lse, dx, dw

    want = [run(i) for i in range(4)]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[i] = run(i)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
