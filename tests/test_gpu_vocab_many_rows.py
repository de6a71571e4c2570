"""Losses over a vocabulary of very many rows (GPU): around the sizes where the rows that have a loss are listed another way."""
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace
from _products import assert_within, loss as loss_ref, loss_backward as backward_ref

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _case(rows, dim=8, vocab=24):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, w = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((rows, dim), (vocab, dim)))
    target = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    h = ac.adacomp_vocab_init(dim, vocab, ac.BF16)
    return x, w, target, g, h


@pytest.mark.parametrize("rows", [16384, 16385, 17000, 1024 * 1024, 1024 * 1024 + 1, 3_000_001])
@pytest.mark.parametrize("which", ["half", "last", "all", "blocks"])
def test_rows(rows, which):
    """Rows with a loss are spread, one alone, all, or in blocks with whole blocks of none."""
    x, w, target, g, h = _case(rows)
    at = torch.arange(rows, device="cuda")
    none = {"half": torch.rand(rows, generator=g, device="cuda") < 0.5, "last": at < rows - 1, "all": at < 0,
            "blocks": at // 5000 % 3 != 1}[which]
    target[none] = -1
    x[none] = NAN
    loss, lse, dx = (torch.full(s, NAN, device="cuda") for s in ((rows,), (rows,), (rows, 8)))
    dx = dx.bfloat16()
    ws = workspace(max(ac.adacomp_vocab_loss_forward_ws_bytes(h, rows), ac.adacomp_vocab_loss_backward_ws_bytes(h, rows))).fill_(255)
    ac.adacomp_vocab_loss_forward(h, x, w, target, loss, lse, ws)
    one = torch.ones(1, device="cuda")
    ac.adacomp_vocab_loss_backward(h, x, w, target, lse, one, ws, dx=dx)
    assert not loss[none].any() and not dx[none].any()
    for part in torch.arange(rows, device="cuda").split(500_000):
        ref, bound = loss_ref(x[part], w, target[part][:, None])
        assert_within(loss[part], ref[0], bound[0], "loss")
        ref, bound = backward_ref(x[part], w, target[part][:, None], lse[part], one.expand(len(part)))
        assert_within(dx[part], ref[0], bound[0], "dx")


def test_lists():
    rows, k = 40_000, 3
    x, w, _, g, h = _case(rows)
    index = torch.randint(-24, 24, (rows, k), generator=g, device="cuda").to(torch.int32)
    logit = torch.randn(rows, k, generator=g, device="cuda")
    loss, lse = (torch.full((rows,), NAN, device="cuda") for _ in range(2))
    ac.adacomp_distill_forward(h, x, w, index, logit, 2.0, loss, lse, workspace(ac.adacomp_distill_forward_ws_bytes(h, rows, k)))
    ref, bound = loss_ref(x, w, index, logit, 2.0)
    assert_within(loss, ref[0], bound[0], "loss")


def test_the_time_grows_as_the_rows_do():
    """Four times the rows take some 4 times as long; where every block of rows counts all those before it, 11 times."""
    times = []
    for rows in (1 << 22, 1 << 24):
        x, w, target, _, h = _case(rows)
        loss, lse = (torch.empty(rows, device="cuda") for _ in range(2))
        ws = workspace(ac.adacomp_vocab_loss_forward_ws_bytes(h, rows))
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        least = float("inf")
        for _ in range(5):
            start.record()
            ac.adacomp_vocab_loss_forward(h, x, w, target, loss, lse, ws)
            end.record()
            end.synchronize()
            least = min(least, start.elapsed_time(end))
        times.append(least)
    assert times[1] < 7 * times[0], times


def test_a_graph_replayed_with_other_rows():
    """The number of rows with a loss, and which, are read when the graph runs."""
    rows = 40_000
    x, w, target, g, h = _case(rows)
    none = torch.rand(rows, generator=g, device="cuda") < 0.3
    wanted = torch.where(none, -1, target)
    ws = workspace(max(ac.adacomp_vocab_loss_forward_ws_bytes(h, rows), ac.adacomp_vocab_loss_backward_ws_bytes(h, rows)))
    loss, lse, one = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.ones(1, device="cuda")
    dx, dw, now = torch.empty_like(x), torch.empty_like(w), torch.full_like(target, -1)

    def step():
        ac.adacomp_vocab_loss_forward(h, x, w, now, loss, lse, ws)
        ac.adacomp_vocab_loss_backward(h, x, w, now, lse, one, ws, dx=dx, dw=dw)

    results = []
    for values in (wanted, target):
        now.copy_(values)
        step()
        results.append([t.clone() for t in (loss, lse, dx, dw)])
    now.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    assert not loss.any() and not dx.any() and not dw.any()
    for values, want in zip((wanted, target), results):
        now.copy_(values)
        graph.replay()
        for a, b in zip((loss, lse, dx, dw), want):
            assert torch.equal(a, b)
