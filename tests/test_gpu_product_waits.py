"""Waits of the products' kernels that run out (GPU): one CTA of every pair copies nothing, so that its pair's products never
begin. The call ends within its bound, what it had not computed is NaN, and later calls are as before."""
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def test_arguments():
    for kind, h in (("linear", ac.adacomp_linear_init(8, 8)), ("vocab", ac.adacomp_vocab_init(8, 8))):
        limit, silent = (getattr(ac.lib(), f"adacomp_{kind}_set_{what}") for what in ("timeout_ns", "fault_injection"))
        assert limit(None, 5) == silent(None, 0) == limit(h.ptr, 0) == limit(h.ptr, 60_000_000_001) == ac.ERR_INVALID_ARG
        assert limit(h.ptr, 1) == limit(h.ptr, 60_000_000_000) == silent(h.ptr, 0xFFFFFFFF) == ac.OK


def _ran_out(kind, h, silent, run):
    """The outputs without the injection, with it, and after it."""
    before = run()
    torch.cuda.synchronize()
    getattr(ac, f"adacomp_{kind}_set_timeout_ns")(h, 20_000_000)  # 20 ms
    getattr(ac, f"adacomp_{kind}_set_fault_injection")(h, silent)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    during = run()
    end.record()
    end.synchronize()
    assert start.elapsed_time(end) < 2000
    getattr(ac, f"adacomp_{kind}_set_fault_injection")(h)
    getattr(ac, f"adacomp_{kind}_set_timeout_ns")(h, 2_000_000_000)
    for a, b in zip(before, run()):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())
    return during


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,din,dout", [(300, 264, 2000), (300, 3000, 520), (2000, 1000, 3000)])
@pytest.mark.parametrize("silent", [0, 1])
def test_linear(silent, rows, din, dout, dt):
    """Sums shorter than the ring of copies, sums in parts, and several tiles a pair."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    x, w, r, dy, z = n(rows, din), n(dout, din), n(rows, dout), n(rows, dout), n(rows, dout)
    h = ac.adacomp_linear_init(din, dout, ac.BF16 if dt == BF16 else ac.F32, ac.ACT_RELU)
    ws = workspace(max(ac.adacomp_linear_forward_ws_bytes(h, rows), ac.adacomp_linear_backward_ws_bytes(h, rows)))

    def run():
        y, pre, dx, dw = (torch.zeros_like(t) for t in (r, r, x, w))
        ac.adacomp_linear_forward(h, x, w, y, ws, residual=r, pre=pre)
        ac.adacomp_linear_backward(h, dy, x, w, ws, pre=z, dx=dx, dw=dw)
        return y, pre, dx, dw

    for t in _ran_out("linear", h, silent, run):
        assert bool(t.isnan().all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("teach", [False, True])
@pytest.mark.parametrize("silent", [0, 1])
def test_vocabulary(silent, teach, dt):
    rows, dim, vocab, k = 600, 300, 4000, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(*s, generator=g, device="cuda").to(dt) for s in ((rows, dim), (vocab, dim)))
    w *= dim ** -0.5
    index = torch.randint(0, vocab, (rows, k), generator=g, device="cuda").to(torch.int32)
    index[::3] = -1
    logit, dloss = torch.randn(rows, k, generator=g, device="cuda"), torch.randn(rows, generator=g, device="cuda")
    target, none = index[:, 0].contiguous(), index[:, 0] < 0
    h = ac.adacomp_vocab_init(dim, vocab, ac.BF16 if dt == BF16 else ac.F32)
    ws = workspace(max(ac.adacomp_distill_forward_ws_bytes(h, rows, k), ac.adacomp_distill_backward_ws_bytes(h, rows, k)))

    def run():
        loss, lse = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
        dx, dw = torch.zeros_like(x), torch.zeros_like(w)
        if teach:
            ac.adacomp_distill_forward(h, x, w, index, logit, 2.0, loss, lse, ws)
            ac.adacomp_distill_backward(h, x, w, index, logit, 2.0, lse, dloss, ws, dx=dx, dw=dw)
        else:
            ac.adacomp_vocab_loss_forward(h, x, w, target, loss, lse, ws)
            ac.adacomp_vocab_loss_backward(h, x, w, target, lse, dloss, ws, dx=dx, dw=dw)
        return loss, lse, dx, dw

    loss, lse, dx, dw = _ran_out("vocab", h, silent, run)
    for t in (loss, lse, dx):
        assert bool(t[~none].isnan().all()) and not t[none].any()
    assert bool(dw.isnan().all())
