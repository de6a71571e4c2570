"""Workspaces of linear layers: none for copies that the kernels of few rows and small matrices do not make (host), and no
call writes past the size that it asks for (GPU)."""
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


@pytest.mark.parametrize("dtype,most", [(ac.F32, 8), (ac.BF16, 16)])
def test_new_tokens_need_no_copy_of_the_weights(dtype, most):
    h = ac.adacomp_linear_init(2048, 50304, dtype)
    for rows in (0, 1, most):
        assert 0 < ac.adacomp_linear_forward_ws_bytes(h, rows) <= 4096
    assert ac.adacomp_linear_forward_ws_bytes(h, most + 1) > 2048 * 50304


@pytest.mark.parametrize("dtype,bytes_each", [(ac.F32, 4), (ac.BF16, 2)])
def test_small_matrices_need_no_copies(dtype, bytes_each):
    """Forward nothing; backward dz (fp32 in four parts of two bytes) and its sums over slices of the rows."""
    h = ac.adacomp_linear_init(128, 250, dtype, ac.ACT_GELU)
    for rows in (17, 64, 200):
        assert 0 < ac.adacomp_linear_forward_ws_bytes(h, rows) <= 4096
        assert ac.adacomp_linear_backward_ws_bytes(h, rows) <= 2 * max(rows, 64) * 256 * bytes_each + 152 * 250 * 4 + 4096


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,din,dout", [(1, 700, 900), (8, 64, 3000), (16, 300, 40), (20, 100, 90), (32, 200, 250), (64, 800, 500),
                                           (300, 130, 77), (700, 515, 333)])
def test_no_call_writes_past_its_size(rows, din, dout, dt):
    g = torch.Generator(device="cuda").manual_seed(rows)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    x, w, dy = n(rows, din), n(dout, din), n(rows, dout)
    h = ac.adacomp_linear_init(din, dout, ac.BF16 if dt == BF16 else ac.F32, ac.ACT_SILU)
    y, pre, dx, dw, db = (torch.empty_like(t) for t in (dy, dy, x, w, w[:, 0].contiguous()))
    results = []
    for fill in (255, 0):
        for need, call in ((ac.adacomp_linear_forward_ws_bytes(h, rows),
                            lambda ws: ac.adacomp_linear_forward(h, x, w, y, ws, pre=pre)),
                           (ac.adacomp_linear_backward_ws_bytes(h, rows),
                            lambda ws: ac.adacomp_linear_backward(h, dy, x, w, ws, pre=pre, dx=dx, dw=dw, db=db))):
            room = torch.full((need + 65536,), fill, dtype=torch.uint8, device="cuda")
            room[need:] = 123
            call(room[:need])
            assert bool((room[need:] == 123).all())
        results.append([t.clone() for t in (y, pre, dx, dw, db)])
    for a, b in zip(*results):
        assert torch.equal(a, b)
