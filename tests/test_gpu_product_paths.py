"""Products of sizes that take each of their ways (GPU): few rows, small matrices alone and split over a cluster, tiles of
every width, sums in parts, both gradients in one launch, and more tiles than go round."""
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace
from _products import assert_within, linear, linear_backward, loss as loss_ref, loss_backward as backward_ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


# rows, inputs, outputs: few rows of long sums; small matrices of one block of terms, of several, and of so few tiles that a
# cluster has one; a row past the small ones; sums in parts; tiles of all widths from 32 to 256 columns; two waves and more of
# tiles; long sums in both gradients
SIZES = [(1, 8200, 48), (16, 4104, 33), (8, 520, 5000), (9, 130, 40), (17, 128, 64), (40, 1000, 60), (60, 2000, 31),
         (257, 700, 300), (70, 6000, 200), (300, 4096, 129), (500, 200, 900), (1300, 96, 1100), (260, 264, 5000),
         (6000, 72, 136), (2500, 1000, 1500), (257, 40, 9000)] + [(600, 136, 32 * i - 3) for i in range(1, 9)]


@DTYPES
@pytest.mark.parametrize("rows,din,dout", SIZES)
def test_linear(rows, din, dout, dt):
    g = torch.Generator(device="cuda").manual_seed(rows)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    x, w, b, r, dy = n(rows, din), n(dout, din) * din ** -0.5, n(dout), n(rows, dout), n(rows, dout)
    kind = ["none", "relu", "gelu", "gelu_tanh", "silu"][(rows + dout) % 5]
    h = ac.adacomp_linear_init(din, dout, ac.BF16 if dt == BF16 else ac.F32, getattr(ac, "ACT_" + kind.upper()))
    y, pre, dx, dw, db = (torch.full_like(t, float("nan")) for t in (r, r, x, w, b))
    ws = workspace(max(ac.adacomp_linear_forward_ws_bytes(h, rows), ac.adacomp_linear_backward_ws_bytes(h, rows))).fill_(255)
    residual = r if rows % 2 else None
    ac.adacomp_linear_forward(h, x, w, y, ws, bias=b, residual=residual, pre=pre)
    ref, bound = linear(x, w, b, residual, kind)
    assert_within(y, ref[0], bound[0], "y")
    assert_within(pre, ref[1], bound[1], "pre")
    ws.fill_(255)
    ac.adacomp_linear_backward(h, dy, x, w, ws, pre=None if kind == "none" else pre, dx=dx, dw=dw, db=db)
    ref, bound = linear_backward(dy, x, w, pre, kind)
    for name, a, v, e in zip(("dx", "dw", "db"), (dx, dw, db), ref, bound):
        assert_within(a, v, e, name)


@DTYPES
@pytest.mark.parametrize("rows,dim,vocab", [(1, 2056, 20000), (512, 64, 20001), (700, 640, 9999), (1500, 96, 30011),
                                            (2600, 40, 700), (300, 3001, 260), (40, 8, 65536)]
                         + [(300, 72, 257 + 37 * i) for i in range(8)])
def test_loss(rows, dim, vocab, dt):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, dim, generator=g, device="cuda").to(dt)
    w = (torch.randn(vocab, dim, generator=g, device="cuda") * 2 * dim ** -0.5).to(dt)
    target = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    target[1::4] = -1
    target[0] = vocab - 1
    dloss = torch.randn(rows, generator=g, device="cuda")
    h = ac.adacomp_vocab_init(dim, vocab, ac.BF16 if dt == BF16 else ac.F32)
    loss, lse = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    dx, dw = torch.full_like(x, float("nan")), torch.full_like(w, float("nan"))
    ws = workspace(max(ac.adacomp_vocab_loss_forward_ws_bytes(h, rows), ac.adacomp_vocab_loss_backward_ws_bytes(h, rows))).fill_(255)
    ac.adacomp_vocab_loss_forward(h, x, w, target, loss, lse, ws)
    ref, bound = loss_ref(x, w, target[:, None])
    assert_within(loss, ref[0], bound[0], "loss")
    assert_within(lse, ref[1], bound[1], "lse")
    ws.fill_(255)
    ac.adacomp_vocab_loss_backward(h, x, w, target, lse, dloss, ws, dx=dx, dw=dw)
    ref, bound = backward_ref(x, w, target[:, None], lse, dloss)
    assert_within(dx, ref[0], bound[0], "dx")
    assert_within(dw, ref[1], bound[1], "dw")


def test_the_error_of_fp32_sums_does_not_grow_with_their_length():
    """Sums of one sign, where truncations in one direction would add up: runs of 256 terms are off by at most 16 steps of
    2^-23 each, in whatever the tensor cores add, and 32 runs' sums by 32 more of 2^-24; 8192 terms in a row would be off by
    up to 512 steps."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = torch.rand(300, 8192, generator=g, device="cuda") + 0.5, torch.rand(400, 8192, generator=g, device="cuda") + 0.5
    h = ac.adacomp_linear_init(8192, 400)
    y = torch.empty(300, 400, device="cuda")
    ac.adacomp_linear_forward(h, x, w, y, workspace(ac.adacomp_linear_forward_ws_bytes(h, 300)))
    ref = x.double() @ w.double().T
    assert ((y.double() - ref).abs() / ref).max() < 16 * 2.0 ** -23 + 32 * 2.0 ** -24 + 2.0 ** -22


@DTYPES
def test_offsets_past_32_bits(dt):
    """Rows so far apart that the last ones begin past 2^32 elements: the bits of rows that are not."""
    rows, din, dout, far = 3000, 72, 136, 1_500_008
    g = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    code = ac.BF16 if dt == BF16 else ac.F32
    x, w, dy = n(rows, din), n(dout, din), n(rows, dout)
    wide = torch.empty(rows * far, dtype=dt, device="cuda").view(rows, far)
    spread = {}
    at = 0
    for name, cols, value in (("x", din, x), ("y", dout, None), ("pre", dout, None), ("dy", dout, dy), ("dx", din, None)):
        spread[name] = wide[:, at:at + cols]
        at += (cols + 7) // 8 * 8
        if value is not None:
            spread[name].copy_(value)
    h = ac.adacomp_linear_init(din, dout, code, ac.ACT_SILU)
    ws = workspace(max(ac.adacomp_linear_forward_ws_bytes(h, rows), ac.adacomp_linear_backward_ws_bytes(h, rows)))
    near = {"y": torch.empty_like(dy), "pre": torch.empty_like(dy), "dx": torch.empty_like(x)}
    grads = []
    for t in (dict(near, x=x, dy=dy), spread):
        dw = torch.empty_like(w)
        ac.adacomp_linear_forward(h, t["x"], w, t["y"], ws, pre=t["pre"])
        ac.adacomp_linear_backward(h, t["dy"], t["x"], w, ws, pre=t["pre"], dx=t["dx"], dw=dw)
        grads.append(dw)
    assert torch.equal(*grads)
    for name in near:
        assert torch.equal(near[name], spread[name]), name
    v = ac.adacomp_vocab_init(din, dout, code)
    target = torch.randint(0, dout, (rows,), generator=g, device="cuda")
    ws = workspace(max(ac.adacomp_vocab_loss_forward_ws_bytes(v, rows), ac.adacomp_vocab_loss_backward_ws_bytes(v, rows)))
    results = []
    for hidden, dx in ((x, torch.empty_like(x)), (spread["x"], spread["dx"])):
        loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        ac.adacomp_vocab_loss_forward(v, hidden, w, target, loss, lse, ws)
        ac.adacomp_vocab_loss_backward(v, hidden, w, target, lse, loss, ws, dx=dx)
        results.append((loss, lse, dx))
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_many_short_rows():
    """So many rows that counting those with a loss takes hundreds of CTAs, and that grids of rows go round."""
    rows, dim, vocab = 600_000, 16, 96
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((rows, dim), (vocab, dim)))
    target = torch.randint(-vocab, vocab, (rows,), generator=g, device="cuda").to(torch.int32)
    v = ac.adacomp_vocab_init(dim, vocab, ac.BF16)
    ws = workspace(max(ac.adacomp_vocab_loss_forward_ws_bytes(v, rows), ac.adacomp_vocab_loss_backward_ws_bytes(v, rows))).fill_(255)
    loss, lse, dx = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x)
    one = torch.ones(1, device="cuda")
    ac.adacomp_vocab_loss_forward(v, x, w, target, loss, lse, ws)
    ac.adacomp_vocab_loss_backward(v, x, w, target, lse, one, ws, dx=dx)
    for part in (slice(0, 20_000), slice(290_000, 310_000), slice(580_000, 600_000)):
        ref, bound = loss_ref(x[part], w, target[part].long()[:, None])
        assert_within(loss[part], ref[0], bound[0], "loss")
        ref, bound = backward_ref(x[part], w, target[part].long()[:, None], lse[part], one.expand(20_000))
        assert_within(dx[part], ref[0], bound[0], "dx")
