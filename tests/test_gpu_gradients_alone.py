"""Gradients of products on the tensor cores (GPU): each one alone has the bits that it has beside the others, also where its
sums are formed in parts."""
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _alone(call, outs, names):
    """`call` with all of the outputs, and with each subset of them."""
    together = {n: torch.full_like(t, float("nan")) for n, t in zip(names, outs)}
    call(**together)
    for bits in range(1, 2 ** len(names) - 1):
        some = {n: torch.full_like(t, float("nan")) for i, (n, t) in enumerate(zip(names, outs)) if bits >> i & 1}
        call(**some)
        for n, t in some.items():
            assert torch.equal(t, together[n]), (sorted(some), n)


@pytest.mark.parametrize("rows,din,dout,dt", [
    (3001, 1001, 777, F32), (2048, 1024, 1024, F32), (1300, 96, 1100, F32), (5000, 72, 200, F32), (100, 3000, 3000, F32),
    (8192, 512, 512, BF16), (1300, 96, 1100, BF16), (20, 2000, 1000, BF16), (20000, 136, 264, BF16), (600, 5000, 700, BF16)])
def test_a_linear_layers(rows, din, dout, dt):
    g = torch.Generator(device="cuda").manual_seed(rows)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    x, w, dy, pre = n(rows, din), n(dout, din), n(rows, dout), n(rows, dout)
    h = ac.adacomp_linear_init(din, dout, ac.BF16 if dt == BF16 else ac.F32, ac.ACT_GELU)
    ws = workspace(ac.adacomp_linear_backward_ws_bytes(h, rows)).fill_(255)
    _alone(lambda **out: ac.adacomp_linear_backward(h, dy, x, w, ws, pre=pre, **out), (x, w, w[:, 0].contiguous()), ("dx", "dw", "db"))


@pytest.mark.parametrize("rows,dim,vocab,dt", [
    (2003, 501, 10007, F32), (300, 3001, 260, F32), (512, 64, 20001, F32), (20, 300, 5000, F32), (2600, 40, 700, BF16),
    (512, 640, 9999, BF16), (9000, 200, 300, BF16), (20, 2000, 5000, BF16), (70_000, 8, 4500, BF16)])
def test_a_vocabularys(rows, dim, vocab, dt):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, w = (torch.randn(*s, generator=g, device="cuda").to(dt) for s in ((rows, dim), (vocab, dim)))
    w *= dim ** -0.5
    target = torch.randint(-vocab // 3, vocab, (rows,), generator=g, device="cuda")
    h = ac.adacomp_vocab_init(dim, vocab, ac.BF16 if dt == BF16 else ac.F32)
    ws = workspace(ac.adacomp_vocab_loss_backward_ws_bytes(h, rows)).fill_(255)
    lse, dloss = torch.full((rows,), 9.0, device="cuda"), torch.randn(rows, generator=g, device="cuda")
    _alone(lambda **out: ac.adacomp_vocab_loss_backward(h, x, w, target, lse, dloss, ws, **out), (x, w), ("dx", "dw"))


def _least_time(call, reps=5, calls=10):
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    least = float("inf")
    for _ in range(reps):
        start.record()
        for _ in range(calls):
            call()
        end.record()
        end.synchronize()
        least = min(least, start.elapsed_time(end))
    return least


@pytest.mark.parametrize("rows", [17, 64])
def test_both_take_no_longer_than_one_after_the_other(rows):
    """A product of few long sums and one of many short ones share a launch: no pair of SMs is left with most tiles of the
    second. (Together they take about 0.8 of the time of both alone; 2.3 when a tile's end was not counted.)"""
    x, w, dy = (torch.randn(*s, device="cuda").bfloat16() for s in ((rows, 2048), (8192, 2048), (rows, 8192)))
    h = ac.adacomp_linear_init(2048, 8192, ac.BF16)
    ws = workspace(ac.adacomp_linear_backward_ws_bytes(h, rows))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    times = [_least_time(lambda: ac.adacomp_linear_backward(h, dy, x, w, ws, **out)) for out in
             ({"dx": dx, "dw": dw}, {"dx": dx, "dw": dw}, {"dx": dx}, {"dw": dw})]
    assert times[1] < 1.3 * (times[2] + times[3])
