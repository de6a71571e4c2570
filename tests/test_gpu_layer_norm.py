"""Layer norm, forward and backward, against the plain form in 64 bits (GPU).

Tolerances are worst-case rounding bounds (tests/_train.py). Sizes cross the edges of the
kernels' variants: widths of one to tens of thousands, odd ones, rows from none, views
with gaps and bases that are aligned to their element alone, and work in place."""
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace
from _train import U, assert_within, norm_backward, norm_forward

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16
CODE = {F: ac.F32, B: ac.BF16}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(gen, *shape, dtype=F, scale=1.0, offset=0.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale + offset).to(dtype)


def _params(gen, dim, wt):
    return _rand(gen, dim, dtype=wt, scale=0.3, offset=1.0), _rand(gen, dim, dtype=wt, scale=0.2)


def _forward(h, x, w, b, y=None):
    rows = x.shape[0]
    y = torch.empty_like(x) if y is None else y
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ac.adacomp_layer_norm_forward(h, x, w, b, y, mean, rstd)
    return y, mean, rstd


def _check_forward(h, x, w, b, y=None):
    ref, bound = norm_forward(x, w, b, EPS)
    got = _forward(h, x, w, b, y)
    for name, g, r, e in zip(("y", "mean", "rstd"), got, ref, bound):
        assert_within(g, r, e, f"{name} {tuple(x.shape)} {x.dtype} {w.dtype}")
    return got


def _backward(h, dy, x, w, mean, rstd, dx=None, bias=True):
    dx = torch.empty_like(x) if dx is None else dx
    dw, db = torch.empty_like(w), torch.empty_like(w) if bias else None
    ws = torch.full((ac.adacomp_layer_norm_backward_ws_bytes(h, x.shape[0]),), 0xff, dtype=torch.uint8, device="cuda")
    ac.adacomp_layer_norm_backward(h, dy, x, w, mean, rstd, dx, dw, db, ws)
    return dx, dw, db


def _check_backward(h, dy, x, w, mean, rstd, dx=None):
    ref, bound = norm_backward(dy, x, w, mean, rstd, w.dtype)
    got = _backward(h, dy, x, w, mean, rstd, dx)
    for name, g, r, e in zip(("dx", "dw", "db"), got, ref, bound):
        assert_within(g, r, e, f"{name} {tuple(x.shape)} {x.dtype} {w.dtype}")
    return got


SIZES = [(1, 1), (5, 2), (3, 7), (9, 31), (64, 32), (33, 33), (257, 100), (1000, 128), (7, 255), (700, 256), (129, 257),
         (65, 511), (300, 512), (31, 1000), (77, 1001), (513, 1024), (20, 2047), (1300, 2048), (6, 2049), (11, 4096),
         (3, 4097), (5, 5000), (2, 8192), (1, 8193), (3, 12345), (2, 16384), (2, 16385), (2, 40000), (1, 100003)]


@pytest.mark.parametrize("xt,wt", [(F, F), (B, F), (B, B), (F, B)])
@pytest.mark.parametrize("rows,dim", SIZES)
def test_forward_and_backward(rows, dim, xt, wt):
    gen = _gen(rows * 131 + dim)
    h = ac.adacomp_layer_norm_init(dim, CODE[xt], CODE[wt], EPS)
    x = _rand(gen, rows, dim, dtype=xt, offset=0.5)
    w, b = _params(gen, dim, wt)
    _, mean, rstd = _check_forward(h, x, w, b)
    _check_backward(h, _rand(gen, rows, dim, dtype=xt, scale=0.1), x, w, mean, rstd)


# both sides of every width at which another variant takes over, in rows of each alignment
WIDTHS = [w + d for w in (128, 256, 512, 1024, 2048, 4096, 8192, 16384) for d in (-1, 0, 2, 8)]


@pytest.mark.parametrize("xt,wt", [(F, F), (B, F), (B, B)])
@pytest.mark.parametrize("dim", WIDTHS)
def test_widths(dim, xt, wt):
    gen, rows = _gen(dim), 309  # more than SMs; below, in test_forward_and_backward, fewer
    h = ac.adacomp_layer_norm_init(dim, CODE[xt], CODE[wt], EPS)
    x = _rand(gen, rows, dim, dtype=xt, offset=0.5)
    w, b = _params(gen, dim, wt)
    _, mean, rstd = _check_forward(h, x, w, b)
    _check_backward(h, _rand(gen, rows, dim, dtype=xt), x, w, mean, rstd)


@pytest.mark.parametrize("rows,dim", [(100_000, 5), (70_000, 64), (20_001, 200), (4096, 768)])
def test_many_rows(rows, dim):
    gen = _gen(rows)
    h = ac.adacomp_layer_norm_init(dim, ac.BF16, ac.F32, EPS)
    x = _rand(gen, rows, dim, dtype=B)
    w, b = _params(gen, dim, F)
    _, mean, rstd = _check_forward(h, x, w, b)
    _check_backward(h, _rand(gen, rows, dim, dtype=B), x, w, mean, rstd)


@pytest.mark.parametrize("dim", [48, 1001, 2048, 20000])
@pytest.mark.parametrize("xt", [F, B])
@pytest.mark.parametrize("shift,gap", [(0, 8), (1, 3), (2, 2), (4, 4), (8, 1)])
def test_strides_and_bases_off_every_alignment(dim, xt, shift, gap):
    """Rows inside a wider buffer that starts `shift` elements in; what lies between the
    rows keeps its bytes."""
    gen, rows = _gen(dim + shift), 37
    h = ac.adacomp_layer_norm_init(dim, CODE[xt], ac.F32, EPS)

    def inside(fill=None):
        flat = torch.full((shift + rows * (dim + gap) + 16,), -7.0, dtype=xt, device="cuda")
        view = flat[shift:shift + rows * (dim + gap)].view(rows, dim + gap)[:, :dim]
        if fill is not None:
            view.copy_(fill)
        return flat, view

    _, x = inside(_rand(gen, rows, dim, dtype=xt, offset=1.0))
    _, dy = inside(_rand(gen, rows, dim, dtype=xt))
    yflat, y = inside()
    w, b = (torch.cat([torch.zeros(1, device="cuda"), t])[1:] for t in _params(gen, dim, F))  # 4-byte aligned only
    _, mean, rstd = _check_forward(h, x, w, b, y)
    dflat, dx = inside()
    _check_backward(h, dy, x, w, mean, rstd, dx)
    for flat, view in ((yflat, y), (dflat, dx)):
        view.fill_(-7.0)
        assert bool((flat == -7.0).all())


def test_rows_of_one_broadcast_row():
    gen, dim = _gen(5), 512
    h = ac.adacomp_layer_norm_init(dim, ac.F32, ac.F32, EPS)
    x = _rand(gen, 1, dim).expand(19, dim)
    w, b = _params(gen, dim, F)
    y = torch.empty(19, dim, device="cuda")
    _, mean, rstd = _check_forward(h, x, w, b, y)
    _check_backward(h, _rand(gen, 1, dim).expand(19, dim), x, w, mean, rstd, y)


@pytest.mark.parametrize("dim", [100, 2048, 30000])
def test_in_place(dim):
    gen, rows = _gen(dim), 65
    h = ac.adacomp_layer_norm_init(dim, ac.BF16, ac.F32, EPS)
    x, dy = _rand(gen, rows, dim, dtype=B), _rand(gen, rows, dim, dtype=B)
    w, b = _params(gen, dim, F)
    y, mean, rstd = _forward(h, x, w, b)
    over = x.clone()
    assert torch.equal(_forward(h, over, w, b, over)[0], y)
    dx, dw, db = _backward(h, dy, x, w, mean, rstd)
    for target in ("dy", "x"):
        dyc, xc = dy.clone(), x.clone()
        got = _backward(h, dyc, xc, w, mean, rstd, dyc if target == "dy" else xc)
        for a, r in zip(got, (dx, dw, db)):
            assert torch.equal(a, r), target


def test_no_rows_and_optional_outputs():
    h = ac.adacomp_layer_norm_init(300, ac.F32, ac.BF16, EPS)
    gen = _gen(0)
    w, b = _params(gen, 300, B)
    none = torch.empty(0, 300, device="cuda")
    ac.adacomp_layer_norm_forward(h, none, w, b, none.clone())
    dx, dw, db = _backward(h, none, none, w, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"))
    assert not dw.any() and not db.any()
    x = _rand(gen, 4, 300)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    ac.adacomp_layer_norm_forward(h, x, w, None, y)
    assert_within(y, norm_forward(x, w, None, EPS)[0][0], norm_forward(x, w, None, EPS)[1][0], "y without a bias")
    _, mean, rstd = _forward(h, x, w, b, y2)
    full = _backward(h, x, x, w, mean, rstd)
    part = _backward(h, x, x, w, mean, rstd, bias=False)
    assert torch.equal(full[0], part[0]) and torch.equal(full[1], part[1])


@pytest.mark.parametrize("xt", [F, B])
def test_constant_offset_large_and_small_rows(xt):
    """A row whose mean is a thousand deviations, an all-equal row (no variance), and rows
    near both ends of the range of the squares."""
    dim = 1000
    gen = _gen(3)
    h = ac.adacomp_layer_norm_init(dim, CODE[xt], ac.F32, EPS)
    x = _rand(gen, 5, dim)
    x[0] = x[0] * 0.125 + 128.0
    x[1] = 3.0
    x[2] *= 1e15
    x[3] *= 1e-15
    x = x.to(xt)
    w, b = _params(gen, dim, F)
    _, mean, rstd = _check_forward(h, x, w, b)
    _check_backward(h, _rand(gen, 5, dim, dtype=xt), x, w, mean, rstd)


@pytest.mark.parametrize("dim", [40, 2048, 20000])
def test_non_finite_values_stay_in_their_row(dim):
    gen = _gen(9)
    h = ac.adacomp_layer_norm_init(dim, ac.F32, ac.F32, EPS)
    x = _rand(gen, 6, dim)
    clean = x.clone()
    w, b = _params(gen, dim, F)
    y0, mean0, rstd0 = _forward(h, clean, w, b)
    x[1, dim // 2], x[4, 0] = float("nan"), float("inf")
    y, mean, rstd = _forward(h, x, w, b)
    for r in range(6):
        if r in (1, 4):
            assert torch.isnan(y[r]).all()
        else:
            assert torch.equal(y[r], y0[r]) and mean[r] == mean0[r] and rstd[r] == rstd0[r]


@pytest.mark.parametrize("dim", [300, 2048])
def test_gradients_against_differences(dim):
    """Directional derivatives of the kernel's own forward pass, in 32 bits. With a step e
    the central difference is off by e^2/6 times a third derivative of order one in units of
    the direction's size, and by the rounding of the two sums over 2 e."""
    gen, rows = _gen(dim), 40
    h = ac.adacomp_layer_norm_init(dim, ac.F32, ac.F32, EPS)
    x, dy = _rand(gen, rows, dim), _rand(gen, rows, dim)
    w, b = _params(gen, dim, F)
    _, mean, rstd = _forward(h, x, w, b)
    grads = _backward(h, dy, x, w, mean, rstd)
    e = 2.0 ** -7
    for k, (base, grad) in enumerate(zip((x, w, b), grads)):
        v = _rand(gen, *base.shape)
        ends = []
        for s in (e, -e):
            args = [x, w, b]
            args[k] = base + s * v
            ends.append((_forward(h, *args)[0].double() * dy.double()).sum())
        got = float((ends[0] - ends[1]) / (2 * e))
        want = float((grad.double() * v.double()).sum())
        scale = float((rows * dim) ** 0.5)  # what a sum of rows * dim terms of random sign comes to
        assert abs(got - want) <= scale * (4 * e * e + 64 * U / e), (k, got, want)


def test_offsets_past_32_bits():
    """Rows 2^30 + 8 elements apart: the last ones lie past 2^31 elements and 2^32 bytes."""
    dim, gap, rows = 96, 2 ** 30 + 8, 4
    gen = _gen(1)
    h = ac.adacomp_layer_norm_init(dim, ac.BF16, ac.F32, EPS)
    flat = torch.empty((rows - 1) * gap + dim, dtype=B, device="cuda")
    x = flat.as_strided((rows, dim), (gap, 1))
    x.copy_(_rand(gen, rows, dim, dtype=B))
    w, b = _params(gen, dim, F)
    keep = x.clone()
    y, mean, rstd = _forward(h, keep, w, b)
    got = _forward(h, x, w, b, torch.empty_like(keep))
    assert all(torch.equal(a, r) for a, r in zip(got, (y, mean, rstd)))
    dy = _rand(gen, rows, dim, dtype=B)
    ref = _backward(h, dy, keep, w, mean, rstd)
    got = _backward(h, dy, x, w, mean, rstd, x)
    assert all(torch.equal(a, r) for a, r in zip(got, ref))


def test_same_inputs_same_bits_also_on_another_stream():
    gen, rows, dim = _gen(2), 3000, 1024
    h = ac.adacomp_layer_norm_init(dim, ac.BF16, ac.F32, EPS)
    x, dy = _rand(gen, rows, dim, dtype=B), _rand(gen, rows, dim, dtype=B)
    w, b = _params(gen, dim, F)
    y, mean, rstd = _forward(h, x, w, b)
    ref = _backward(h, dy, x, w, mean, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            assert torch.equal(_forward(h, x, w, b)[0], y)
            assert all(torch.equal(a, r) for a, r in zip(_backward(h, dy, x, w, mean, rstd), ref))
    side.synchronize()


def test_capture_in_a_graph():
    gen, rows, dim = _gen(4), 128, 768
    h = ac.adacomp_layer_norm_init(dim, ac.BF16, ac.F32, EPS)
    x, dy = _rand(gen, rows, dim, dtype=B), _rand(gen, rows, dim, dtype=B)
    w, b = _params(gen, dim, F)
    y, mean, rstd = _forward(h, x, w, b)
    ref = _backward(h, dy, x, w, mean, rstd)
    out = [torch.zeros_like(t) for t in (y, mean, rstd, *ref)]
    ws = workspace(ac.adacomp_layer_norm_backward_ws_bytes(h, rows))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ac.adacomp_layer_norm_forward(h, x, w, b, out[0], out[1], out[2])
        ac.adacomp_layer_norm_backward(h, dy, x, w, out[1], out[2], out[3], out[4], out[5], ws)
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, r) for a, r in zip(out, (y, mean, rstd, *ref)))
