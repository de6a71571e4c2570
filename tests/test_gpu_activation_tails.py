"""Activations and slopes where they vanish (GPU): far below 0 they are right relative to themselves, not only to z."""
import math

import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace
from _products import OUT, U

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
A, B = math.sqrt(2 / math.pi), 0.044715


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _plain(z, kind):
    """In 64 bits: the activation, its slope and the magnitudes of the slope's terms, and an error relative to each of them
    that fp32 steps have (squares and exponents are off by some units, which the exponential multiplies by its argument)."""
    if kind == "gelu":
        c, bell = 0.5 * torch.special.erfc(-z / math.sqrt(2)), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z * c, c + z * bell, c + z.abs() * bell, (2 * z * z + 16) * U
    if kind == "gelu_tanh":
        u = A * (z + B * z ** 3)
        s, rise = torch.sigmoid(2 * u), 2 * z * torch.sigmoid(-2 * u) * A * (1 + 3 * B * z * z)
        return z * s, s * (1 + rise), s * (1 + rise.abs()), (16 * u.abs() + 32) * U
    g = torch.sigmoid(z)
    return z * g, g * (1 + z * torch.sigmoid(-z)), g * (1 + z.abs()), torch.full_like(z, 32 * U)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind,lowest", [("gelu", -13.0), ("gelu_tanh", -10.0), ("silu", -85.0)])
@pytest.mark.parametrize("rows", [1, 12, 300])
def test_far_below_zero(rows, kind, lowest, dt):
    """Down to where results leave the normal numbers. bf16 layers' quick functions are off by 2^-12 of the value at most
    (erfc's fit 7.3e-5, the exponential 4e-5 at its argument of -88, fp32 steps less), the results by half a step more."""
    z = torch.linspace(lowest, 0.0, 1024, device="cuda").to(dt)
    h = ac.adacomp_linear_init(1, 1024, ac.BF16 if dt == BF16 else ac.F32, getattr(ac, "ACT_" + kind.upper()))
    x, w = torch.ones(rows, 1, dtype=dt, device="cuda"), z[:, None].contiguous()
    y, pre = (torch.full((rows, 1024), math.nan, dtype=dt, device="cuda") for _ in range(2))
    ac.adacomp_linear_forward(h, x, w, y, workspace(ac.adacomp_linear_forward_ws_bytes(h, rows)), pre=pre)
    assert torch.equal(pre, z.expand_as(pre))
    # one row's gradient of the bias is its slope
    dy, db = torch.zeros_like(y), torch.full((1024,), math.nan, dtype=dt, device="cuda")
    dy[rows // 2] = 1.0
    ac.adacomp_linear_backward(h, dy, x, w, workspace(ac.adacomp_linear_backward_ws_bytes(h, rows)), pre=pre, db=db)
    value, slope, size, rel = _plain(z.double(), kind)
    rel = rel + (2.0 ** -12 if dt == BF16 else 0.0)
    for name, got, ref, err in (("y", y, value, rel * value.abs()), ("slope", db, slope, rel * size)):
        bound = err * (1 + OUT[dt]) + OUT[dt] * ref.abs() + 2.0 ** -126  # numbers below the normal ones may be flushed
        over = ((got.double() - ref).abs() - bound).max(0).values if got.dim() > 1 else (got.double() - ref).abs() - bound
        at = int(over.argmax())
        assert float(over.max()) <= 0, (name, float(z[at]), got[..., at].flatten()[:1].tolist(), float(ref[at]))


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("rows", [1, 300])
def test_far_from_zero(rows, kind, dt):
    """Values whose squares or cubes overflow: the activation is z or 0, its slope 1 or 0."""
    z = torch.tensor([s * 10.0 ** e for s in (1, -1) for e in (3, 6, 10, 14, 19, 20, 30, 38)], device="cuda").to(dt).repeat(64)
    n = z.numel()
    h = ac.adacomp_linear_init(1, n, ac.BF16 if dt == BF16 else ac.F32, getattr(ac, "ACT_" + kind.upper()))
    x, w = torch.ones(rows, 1, dtype=dt, device="cuda"), z[:, None].contiguous()
    y, pre = (torch.full((rows, n), math.nan, dtype=dt, device="cuda") for _ in range(2))
    ac.adacomp_linear_forward(h, x, w, y, workspace(ac.adacomp_linear_forward_ws_bytes(h, rows)), pre=pre)
    on = (z > 0) | (kind == "none")
    assert torch.equal(y, torch.where(on, z, 0.0).expand_as(y))
    dy, db = torch.zeros_like(y), torch.full((n,), math.nan, dtype=dt, device="cuda")
    dy[rows // 2] = 1.0
    ac.adacomp_linear_backward(h, dy, x, w, workspace(ac.adacomp_linear_backward_ws_bytes(h, rows)), pre=pre, db=db)
    assert torch.equal(db, on.to(dt))
