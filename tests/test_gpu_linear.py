"""Linear layers (GPU): forward and backward pass against plain forms in 64 bits, within bounds derived
from the operations."""
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace
from _products import act, assert_within, linear, linear_backward, strided

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
ACTS = {"none": ac.ACT_NONE, "relu": ac.ACT_RELU, "gelu": ac.ACT_GELU, "gelu_tanh": ac.ACT_GELU_TANH,
        "silu": ac.ACT_SILU}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _code(dt):
    return ac.BF16 if dt == BF16 else ac.F32


def _inputs(rows, din, dout, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (n(rows, din).to(dt), (n(dout, din) * din ** -0.5).to(dt), n(dout).to(dt), n(rows, dout).to(dt),
            n(rows, dout).to(dt))


class Layer:
    def __init__(self, din, dout, dt, kind):
        self.h, self.din, self.dout, self.dt, self.kind = ac.adacomp_linear_init(din, dout, _code(dt), ACTS[kind]), din, dout, dt, kind

    def forward(self, x, w, bias=None, residual=None, y=None, pre=None, ws=None):
        rows = x.shape[0]
        y = torch.full((rows, self.dout), float("nan"), dtype=self.dt, device="cuda") if y is None else y
        pre = torch.full((rows, self.dout), float("nan"), dtype=self.dt, device="cuda") if pre is None else pre
        ws = workspace(ac.adacomp_linear_forward_ws_bytes(self.h, rows)).fill_(255) if ws is None else ws
        ac.adacomp_linear_forward(self.h, x, w, y, ws, bias=bias, residual=residual, pre=pre)
        return y, pre

    def backward(self, dy, x, w, pre, dx=None, dw=None, ws=None):
        rows = dy.shape[0]
        dx = torch.full((rows, self.din), float("nan"), dtype=self.dt, device="cuda") if dx is None else dx
        dw = torch.full((self.dout, self.din), float("nan"), dtype=self.dt, device="cuda") if dw is None else dw
        db = torch.full((self.dout,), float("nan"), dtype=self.dt, device="cuda")
        ws = workspace(ac.adacomp_linear_backward_ws_bytes(self.h, rows)).fill_(255) if ws is None else ws
        ac.adacomp_linear_backward(self.h, dy, x, w, ws, pre=pre, dx=dx, dw=dw, db=db)
        return dx, dw, db


def _check(layer, x, w, bias, residual, dy, forward_only=False):
    y, pre = layer.forward(x, w, bias, residual)
    ref, bound = linear(x, w, bias, residual, layer.kind)
    assert_within(y, ref[0], bound[0], "y")
    assert_within(pre, ref[1], bound[1], "pre")
    if forward_only:
        return
    got = layer.backward(dy, x, w, None if layer.kind == "none" else pre)
    ref, bound = linear_backward(dy, x, w, pre, layer.kind)
    for name, a, r, b in zip(("dx", "dw", "db"), got, ref, bound):
        assert_within(a, r, b, name)


SIZES = [(1, 1, 1), (1, 64, 100), (1, 2048, 1000), (2, 33, 7), (3, 800, 500), (8, 100, 333), (16, 256, 1024),
         (17, 1001, 130), (33, 72, 256), (64, 800, 500), (127, 64, 129), (128, 512, 256), (129, 65, 257),
         (300, 301, 302), (256, 1024, 768), (1000, 200, 40), (513, 8, 1031)]


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,din,dout", SIZES)
def test_sizes(rows, din, dout, dt):
    kind = ["none", "relu", "gelu", "gelu_tanh", "silu"][(rows + din + dout) % 5]
    x, w, b, r, dy = _inputs(rows, din, dout, dt)
    _check(Layer(din, dout, dt, kind), x, w, b, r, dy)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", list(ACTS))
@pytest.mark.parametrize("rows", [1, 5, 130])
def test_activations(rows, kind, dt):
    """Values from far below to far above 0, with and without bias and residual."""
    x, w, b, r, dy = _inputs(rows, 96, 200, dt, 3)
    x = x * torch.logspace(-3, 1.3, 96, device="cuda").to(dt)
    layer = Layer(96, 200, dt, kind)
    _check(layer, x, w, b, None, dy)
    _check(layer, x, w, None, r, dy)
    _check(layer, x, w, None, None, dy, True)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (8, 0), (3, 5), (8, 8)])
@pytest.mark.parametrize("rows", [1, 4, 40, 200])
def test_strides_and_alignment(rows, pad, shift, dt):
    """Every matrix strided, off alignment and inside a larger buffer of which nothing else changes."""
    din, dout = 136, 264
    x, w, b, r, dy = _inputs(rows, din, dout, dt, 4)
    place = lambda t: strided(t, pad, shift)  # noqa: E731
    flat = torch.full((dout + 9,), float("nan"), dtype=dt, device="cuda")
    bias = flat[shift:shift + dout].copy_(b)
    layer = Layer(din, dout, dt, "silu")
    buffers = [place(torch.zeros(n, k, dtype=dt, device="cuda")) for n, k in
               ((rows, dout), (rows, dout), (rows, din), (dout, din))]
    y, pre = layer.forward(place(x), place(w), bias, place(r), buffers[0], buffers[1])
    ref, bound = linear(x, w, b, r, "silu")
    assert_within(y, ref[0], bound[0], "y")
    got = layer.backward(place(dy), place(x), place(w), pre, buffers[2], buffers[3])
    ref, bound = linear_backward(dy, x, w, pre, "silu")
    for name, a, v, e in zip(("dx", "dw", "db"), got, ref, bound):
        assert_within(a, v, e, name)
    for t in buffers:
        base = t._base if t._base is not None else t
        whole = torch.as_strided(base, (base.numel(),), (1,), 0)
        inside = torch.zeros_like(whole, dtype=torch.bool)
        torch.as_strided(inside, t.shape, t.stride(), t.storage_offset()).fill_(True)
        assert torch.isnan(whole[~inside]).all()


@pytest.mark.parametrize("rows", [1, 9, 70, 300])
def test_fp32_is_not_rounded_to_fewer_bits(rows):
    """Products by a selection, and sums of whole numbers below 2^24, are exact."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randint(-2 ** 24, 2 ** 24, (rows, 200), generator=g, device="cuda").float()
    at = torch.randint(0, 200, (150,), generator=g, device="cuda")
    w = torch.zeros(150, 200, device="cuda")
    w[torch.arange(150, device="cuda"), at] = -2.0
    layer = Layer(200, 150, F32, "none")
    assert torch.equal(layer.forward(x, w)[0], -2.0 * x[:, at])
    dx, dw, _ = layer.backward(torch.ones(rows, 150, device="cuda"), x.sign() * 4095, w, None)
    assert torch.equal(dx.double(), torch.ones(rows, 150, device="cuda").double() @ w.double())
    assert torch.equal(dw.double(), torch.ones(150, rows, device="cuda").double() @ (x.sign() * 4095).double())
    x = torch.randint(-4095, 4096, (rows, 16), generator=g, device="cuda").float()
    w = torch.randint(-255, 256, (150, 16), generator=g, device="cuda").float()
    assert torch.equal(Layer(16, 150, F32, "none").forward(x, w)[0].double(), x.double() @ w.double().T)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_magnitudes(dt):
    """From 2^-60 to 2^60: no part of a number overflows or is lost."""
    x, w, _, _, dy = _inputs(140, 90, 70, dt, 6)
    for a, b in ((60, -60), (-60, 60), (-60, -60), (40, 60)):
        _check(Layer(90, 70, dt, "none"), x * 2.0 ** a, w * 2.0 ** b, None, None, dy)
    big = torch.full((3, 4), 3.3e38, dtype=dt, device="cuda")
    one = torch.tensor([[0.5, 0, 0, 0], [0, -1, 0, 0]], dtype=dt, device="cuda")
    y, _ = Layer(4, 2, dt, "none").forward(big, one)
    assert torch.equal(y, torch.stack([big[:, 0] * 0.5, -big[:, 0]], 1))


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [2, 20, 150])
def test_values_that_are_not_finite(rows, dt):
    """They reach the results that depend on them, and no others; infinities are as in plain arithmetic."""
    x, w, b, r, dy = _inputs(rows, 70, 90, dt, 7)
    inf = float("inf")
    x[0, 3], x[1, 5], w[11, 8] = inf, float("nan"), -inf
    w[12, 3] = 0.0
    r[0, 20] = -inf
    y, _ = Layer(70, 90, dt, "none").forward(x, w, b, r)
    ref = x.double() @ w.double().T + b.double() + r.double()
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    assert torch.equal(torch.isposinf(y), torch.isposinf(ref)) and torch.equal(torch.isneginf(y), torch.isneginf(ref))
    x, w = _inputs(rows, 70, 90, dt, 8)[:2]
    dy[0, 4], dy[1, 9], x[0, 1] = inf, float("nan"), -inf
    dx, dw, db = Layer(70, 90, dt, "none").backward(dy, x, w, None)
    for got, ref in ((dx, dy.double() @ w.double()), (dw, dy.double().T @ x.double()), (db, dy.double().sum(0))):
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.isinf(got), torch.isinf(ref))
        assert torch.equal(got[torch.isinf(got)].sign().double(), ref[torch.isinf(ref)].sign())
    for kind in ACTS:
        z = torch.tensor([[inf, -inf, float("nan"), 0.0]], dtype=dt, device="cuda")
        one = torch.ones(1, 1, dtype=dt, device="cuda")
        y, pre = Layer(1, 4, dt, kind).forward(one, z.T.contiguous())
        assert torch.equal(torch.isnan(pre), torch.isnan(z)) and float(y[0, 0]) == inf and bool(torch.isnan(y[0, 2]))
        assert float(y[0, 3]) == 0.0


@pytest.mark.parametrize("rows,din,dout", [(1, 1, 1), (1, 700, 3), (2, 40, 900), (20, 520, 1000), (32, 1000, 2000), (33, 1000, 2000)])
def test_gradients_of_few_bf16_rows_are_not_rounded_twice(rows, din, dout):
    """dz of up to 32 rows is taken in two parts, 2^-15 of it apart from its value, and slopes are off by 128 * 2^-24, so that
    little but the results' own rounding is left; of more rows it is rounded to 2^-8."""
    x, w, b, _, dy = _inputs(rows, din, dout, BF16, 14)
    layer = Layer(din, dout, BF16, "silu")
    _, pre = layer.forward(x, w, b)
    dx, dw, _ = layer.backward(dy, x, w, pre)
    dz = dy.double() * act(pre.double(), "silu")[1]
    e = dz.abs() * (2.0 ** -15 if rows <= 32 else 2.0 ** -8) + dy.double().abs() * 2.0 ** -16
    for got, ref, size in ((dx, dz @ w.double(), e @ w.double().abs()), (dw, dz.T @ x.double(), e.T @ x.double().abs())):
        assert_within(got, ref, ref.abs() * 2.0 ** -8 + size * 1.01, "gradient")


@pytest.mark.parametrize("rows", [3, 32, 40])
def test_infinite_factors_of_a_gradient(rows):
    """bf16, with an activation: an infinite weight or input makes what it meets infinite with the gradient's sign."""
    for din, dout in ((40, 60), (520, 2000)):
        x, w, _, _, dy = _inputs(rows, din, dout, BF16, 15)
        x[1, 2], w[3, 4] = float("inf"), float("-inf")
        dy[:, 3], dy[1, 5] = 1.0, -2.0
        pre = torch.full_like(dy, 30.0)  # slopes of 1, exactly
        dx, dw, _ = Layer(din, dout, BF16, "silu").backward(dy, x, w, pre)
        ref = dy.double() @ w.double(), dy.double().T @ x.double()
        for got, want in zip((dx, dw), ref):
            assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))
            assert torch.equal(got[torch.isinf(got)].sign().double(), want[torch.isinf(want)].sign())


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_one_row_for_all(dt):
    """A stride of 0 between rows, of x, the weights, the residual and dy."""
    x, w, b, r, dy = _inputs(1, 40, 50, dt, 9)
    rows = 37
    wide = lambda t: t.expand(rows, t.shape[1])  # noqa: E731
    layer = Layer(40, 50, dt, "gelu")
    y, pre = layer.forward(wide(x), w, b, wide(r))
    assert torch.equal(y, y[:1].expand_as(y))
    ref, bound = linear(wide(x), w, b, wide(r), "gelu")
    assert_within(y, ref[0], bound[0], "y")
    ref, bound = linear_backward(wide(dy), wide(x), w, pre, "gelu")
    for a, v, e in zip(layer.backward(wide(dy), wide(x), w, pre), ref, bound):
        assert_within(a, v, e, "gradients of one row for all")
    alike = w[:1].expand(50, 40)
    y, _ = Layer(40, 50, dt, "none").forward(x, alike)
    ref, bound = linear(x, alike, None, None, "none")
    assert_within(y, ref[0], bound[0], "one weight row for all")


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_no_rows(dt):
    layer = Layer(30, 20, dt, "relu")
    x, w = torch.empty(0, 30, dtype=dt, device="cuda"), torch.ones(20, 30, dtype=dt, device="cuda")
    layer.forward(x, w)
    dx, dw, db = layer.backward(torch.empty(0, 20, dtype=dt, device="cuda"), x, w, torch.empty(0, 20, dtype=dt, device="cuda"))
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [3, 150])
def test_only_what_is_wanted(rows, dt):
    """Each gradient alone is the one of all together, and an output in the residual's place."""
    x, w, b, r, dy = _inputs(rows, 104, 88, dt, 10)
    layer = Layer(104, 88, dt, "gelu_tanh")
    y, pre = layer.forward(x, w, b, r)
    dx, dw, db = layer.backward(dy, x, w, pre)
    ws = workspace(ac.adacomp_linear_backward_ws_bytes(layer.h, rows))
    for name, want in (("dx", dx), ("dw", dw), ("db", db)):
        got = torch.empty_like(want)
        ac.adacomp_linear_backward(layer.h, dy, x if name == "dw" else None, w if name == "dx" else None, ws, pre=pre,
                                   **{name: got})
        assert torch.equal(got, want), name
    again = r.clone()
    ac.adacomp_linear_forward(layer.h, x, w, again, workspace(ac.adacomp_linear_forward_ws_bytes(layer.h, rows)), bias=b,
                              residual=again)
    assert torch.equal(again, y)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 12, 260])
def test_determinism_streams_and_graphs(rows, dt):
    """The same bits again, on another stream, and from a replayed graph with new inputs in place."""
    x, w, b, r, dy = _inputs(rows, 264, 520, dt, 11)
    layer = Layer(264, 520, dt, "gelu")
    first = (*layer.forward(x, w, b, r), *layer.backward(dy, x, w, layer.forward(x, w, b, r)[1]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, pre = layer.forward(x, w, b, r)
        second = (y, pre, *layer.backward(dy, x, w, pre))
    torch.cuda.current_stream().wait_stream(side)
    for a, c in zip(first, second):
        assert torch.equal(a, c)
    ws = workspace(max(ac.adacomp_linear_forward_ws_bytes(layer.h, rows), ac.adacomp_linear_backward_ws_bytes(layer.h, rows)))
    xs = torch.zeros_like(x)
    out = [torch.empty_like(t) for t in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(xs, w, b, r, out[0], out[1], ws)
        ac.adacomp_linear_backward(layer.h, dy, xs, w, ws, pre=out[1], dx=out[2], dw=out[3], db=out[4])
    for _ in range(2):
        xs.copy_(x)
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        for a, c in zip(first, out):
            assert torch.equal(a, c)


@pytest.mark.parametrize("kind", list(ACTS))
def test_gradients_against_differences(kind):
    """In fp32: a step of h along a direction changes the sum of dy * y by h times the gradients' product with
    it. The second difference is left out: h^2 |y''| / 6 of a sum whose third derivatives are below 3."""
    x, w, b, _, dy = _inputs(20, 24, 28, F32, 12)
    if kind == "relu":
        x = x.abs()
        w = (w.abs() + 0.05) * torch.where(torch.arange(28, device="cuda") % 2 == 0, 1.0, -1.0)[:, None]
        b = torch.zeros_like(b)  # no value comes near 0, where the slope jumps
    layer = Layer(24, 28, F32, kind)
    _, pre = layer.forward(x, w, b)
    dx, dw, db = (t.double() for t in layer.backward(dy, x, w, pre))
    g = torch.Generator(device="cuda").manual_seed(13)
    for gradient, value in ((dx, x), (dw, w), (db, b)):
        way = torch.randn(value.shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4

        def total(s):
            at = [t.double() + s * way if t is value else t.double() for t in (x, w, b)]
            return (dy.double() * act(at[0] @ at[1].T + at[2], kind)[0]).sum()

        slope = (total(h) - total(-h)) / (2 * h)
        want = (gradient * way).sum()
        size = (gradient.abs() * way.abs()).sum()
        assert abs(slope - want) < 1e-5 * size + 1e-4, (kind, float(slope), float(want))
