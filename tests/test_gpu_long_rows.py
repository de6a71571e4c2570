"""Layer norm over rows of millions of elements (GPU), forward and backward, against the plain
form in 64 bits with bounds that do not grow with the row: no sum adds more than RUN terms in
sequence in 32 bits. Rows of nearly equal values, whose sums round one way throughout."""
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace
from _train import OUT, U, assert_within

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16
CODE = {F: ac.F32, B: ac.BF16}
EPS = 1e-5
RUN = 256 + 16  # terms of a run, and the sums over lanes, warps and runs with the roundings around them


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _rand(gen, *shape, dtype=F, scale=1.0, offset=0.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale + offset).to(dtype)


@pytest.mark.parametrize("xt,dim,offset,scale", [(F, 2 ** 23 + 3, 0.1, 1e-5), (F, 2 ** 22, 7.3, 1e-4),
                                                 (B, 2 ** 23 + 8, 0.1, 1e-2), (B, 2 ** 22 + 1, 7.3, 0.5)])
def test_long_rows_with_an_offset(xt, dim, offset, scale):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(dim)
    rows = 2
    h = ac.adacomp_layer_norm_init(dim, CODE[xt], ac.F32, EPS)
    x = _rand(gen, rows, dim, dtype=xt, scale=scale, offset=offset)
    w, b = _rand(gen, dim, scale=1e-5, offset=1.0), _rand(gen, dim, scale=0.1)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ac.adacomp_layer_norm_forward(h, x, w, b, y, mean, rstd)
    xd, wd, bd = x.double(), w.double(), b.double()
    m = xd.mean(1, keepdim=True)
    dev = xd - m
    var = (dev * dev).mean(1, keepdim=True)
    r = (var + EPS).rsqrt()
    e_m = RUN * U * xd.abs().mean(1, keepdim=True)
    e_dev = e_m + U * (xd.abs() + m.abs())
    e_var = (2 * dev.abs() * e_dev + e_dev * e_dev).mean(1, keepdim=True) + RUN * U * var
    assert bool((e_var < 0.1 * (var + EPS)).all())
    e_r = (var + EPS - e_var).rsqrt() - r + 4 * U * r
    assert_within(mean, m[:, 0], e_m[:, 0], "mean")
    assert_within(rstd, r[:, 0], e_r[:, 0], "rstd")
    want = dev * r * wd + bd
    e_y = wd.abs() * (e_dev * (r + e_r) + dev.abs() * e_r) + 4 * U * (want.abs() + bd.abs())
    assert_within(y, want, e_y + OUT[xt] * (want.abs() + e_y), "y")

    # the backward pass, from these statistics: dy with an offset, so that sum(g) is large
    dy = _rand(gen, rows, dim, dtype=xt, scale=1e-5, offset=0.1)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    ws = workspace(ac.adacomp_layer_norm_backward_ws_bytes(h, rows))
    ac.adacomp_layer_norm_backward(h, dy, x, w, mean, rstd, dx, dw, db, ws)
    m, r, g = mean.double()[:, None], rstd.double()[:, None], dy.double() * wd
    xh = (xd - m) * r
    e_xh = r * U * (xd.abs() + m.abs()) + 3 * U * xh.abs()
    s0, s1 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    want = r * (g - s0 - xh * s1)
    e_s0 = RUN * U * g.abs().mean(1, keepdim=True)
    e_s1 = RUN * U * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * e_xh).mean(1, keepdim=True)
    e = r * (6 * U * (g.abs() + s0.abs() + (xh * s1).abs()) + e_s0 + xh.abs() * e_s1 + e_xh * s1.abs() + e_xh * e_s1)
    assert_within(dx, want, e + OUT[xt] * (want.abs() + e), "dx")
