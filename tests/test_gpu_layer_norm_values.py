"""Layer norm's backward pass with values that are not finite (GPU): they reach the row that has
them and the columns of the weight's and bias's gradients that depend on them, and no other bit."""
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16
CODE = {F: ac.F32, B: ac.BF16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


# a group of lanes, a warp, some warps and all of a CTA's per row; strips of columns; rows off alignment
@pytest.mark.parametrize("xt", [F, B])
@pytest.mark.parametrize("rows,dim", [(9, 40), (400, 63), (33, 512), (31, 1001), (309, 2048), (160, 4097), (170, 8192),
                                      (5, 9001), (7, 20000)])
def test_backward(rows, dim, xt):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(dim)
    h = ac.adacomp_layer_norm_init(dim, CODE[xt], ac.F32)
    x, dy = (torch.randn(rows, dim, generator=gen, device="cuda").to(xt) for _ in range(2))
    w = torch.randn(dim, generator=gen, device="cuda")

    def run(x, dy):
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        dw, db = torch.empty_like(w), torch.empty_like(w)
        ws = workspace(ac.adacomp_layer_norm_backward_ws_bytes(h, rows))
        ac.adacomp_layer_norm_forward(h, x, w, None, y, mean, rstd)
        ac.adacomp_layer_norm_backward(h, dy, x, w, mean, rstd, dx, dw, db, ws)
        return dx, dw, db

    clean = run(x, dy)
    assert all(bool(torch.isfinite(t).all()) for t in clean)
    # in dy: its row of dx, and its column of dw and db
    bad = {rows - 1: (0, float("nan")), rows // 2: (dim - 1, float("inf")), 0: (dim // 2, -float("inf"))}
    dirty = dy.clone()
    for r, (c, v) in bad.items():
        dirty[r, c] = v
    dx, dw, db = run(x, dirty)
    keep, cols = torch.ones(rows, dtype=torch.bool, device="cuda"), torch.ones(dim, dtype=torch.bool, device="cuda")
    keep[list(bad)], cols[[c for c, _ in bad.values()]] = False, False
    assert torch.equal(dx[keep], clean[0][keep]) and not bool(torch.isfinite(dx[~keep]).any())
    for got, want in ((dw, clean[1]), (db, clean[2])):
        assert torch.equal(got[cols], want[cols]) and not bool(torch.isfinite(got[~cols]).any())
    assert db[dim - 1] == float("inf") and db[dim // 2] == -float("inf") and bool(db[0].isnan())
    # in x: its row's statistics and so that row of dx, and every column of dw; db does not depend on x
    for v in (float("nan"), float("inf")):
        dirty = x.clone()
        dirty[rows // 2, dim // 3] = v
        dx, dw, db = run(dirty, dy)
        keep[:] = True
        keep[rows // 2] = False
        assert torch.equal(dx[keep], clean[0][keep]) and bool(dx[~keep].isnan().all())
        assert bool(dw.isnan().all()) and torch.equal(db, clean[2])
