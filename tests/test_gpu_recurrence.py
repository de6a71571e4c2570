"""The gated linear recurrence, forward and backward, against the plain form in 64 bits
(GPU): step by step, with worst-case bounds that follow the recurrence (tests/_train.py).
Steps cross the edges of the chunks that a kernel splits the sequence into."""
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built
from _train import U, assert_within, recurrence

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16
CODE = {F: ac.F32, B: ac.BF16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(gen, *shape, dtype=F, scale=1.0, offset=0.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale + offset).to(dtype)


def _inputs(seed, batch, steps, ch, dt, gate=2.0):
    gen = _gen(seed)
    return (_rand(gen, batch, steps, ch, dtype=dt, offset=gate), _rand(gen, batch, steps, ch, dtype=dt),
            _rand(gen, batch, ch), _rand(gen, batch, steps, ch, dtype=dt), _rand(gen, batch, ch))


def _carry(h, batch, steps):
    n = ac.adacomp_recurrence_carry_bytes(h, batch, steps) // 4
    return torch.full((n,), float("nan"), device="cuda")


def _run(z, x, h0, lengths, dy, dh_last, dz=None, dx=None, y=None):
    batch, steps, ch = z.shape
    h = ac.adacomp_recurrence_init(ch, CODE[z.dtype])
    new = lambda: torch.full((batch, steps, ch), -9.0, dtype=z.dtype, device="cuda")  # noqa: E731
    y = new() if y is None else y
    dz = new() if dz is None else dz
    dx = new() if dx is None else dx
    h_last, dh0 = torch.empty(batch, ch, device="cuda"), torch.empty(batch, ch, device="cuda")
    carry = _carry(h, batch, steps)
    ac.adacomp_recurrence_forward(h, z, x, y, h0=h0, lengths=lengths, h_last=h_last, carry=carry)
    ac.adacomp_recurrence_backward(h, z, x, dy, carry, dz, dx, lengths=lengths, dh_last=dh_last, dh0=dh0)
    return y, h_last, dz, dx, dh0


def _check(got, z, x, h0, lengths, dy, dh_last):
    ref, bound = recurrence(z, x, h0, lengths, dy, dh_last)
    for name, g, r, e in zip(("y", "h_last", "dz", "dx", "dh0"), got, ref, bound):
        assert_within(g, r, e, f"{name} {tuple(z.shape)} {z.dtype}")


SIZES = [(1, 1, 1), (3, 1, 70), (64, 1, 1024), (2, 2, 3), (1, 7, 33), (5, 15, 64), (2, 16, 65), (3, 17, 2), (1, 31, 130),
         (2, 63, 32), (2, 64, 64), (1, 65, 66), (2, 127, 5), (2, 128, 96), (1, 129, 63), (1, 255, 64), (3, 257, 40),
         (1, 512, 31), (1, 1000, 129), (1, 1023, 64), (2, 1025, 68), (1, 2049, 7), (1, 4500, 1), (20, 300, 200),
         (300, 40, 33), (2, 130, 4096), (21, 9, 1001), (40, 16, 700), (25, 17, 900), (30, 32, 800), (2, 3, 9)]


@pytest.mark.parametrize("dt", [F, B])
@pytest.mark.parametrize("batch,steps,ch", SIZES)
def test_forward_and_backward(batch, steps, ch, dt):
    z, x, h0, dy, dh = _inputs(batch + steps * 7 + ch, batch, steps, ch, dt)
    _check(_run(z, x, h0, None, dy, dh), z, x, h0, None, dy, dh)


@pytest.mark.parametrize("dt", [F, B])
@pytest.mark.parametrize("batch,steps,ch", [(7, 200, 37), (6, 1300, 64), (9, 20, 130)])
def test_lengths_and_what_lies_past_them(batch, steps, ch, dt):
    """Whole, empty, negative and overlong lengths; NaN past the end reaches nothing."""
    z, x, h0, dy, dh = _inputs(batch, batch, steps, ch, dt)
    lengths = torch.tensor(([steps, 0, 1, steps - 1, steps // 2, -3, steps + 100, 129, 128] * 2)[:batch],
                           dtype=torch.int32, device="cuda")
    ends = lengths.clamp(0, steps)
    gone = torch.arange(steps, device="cuda")[None, :] >= ends[:, None]
    for t in (z, x, dy):
        t[gone] = float("nan")
    got = _run(z, x, h0, lengths, dy, dh)
    _check(got, z, x, h0, lengths, dy, dh)
    for k in (0, 2, 3):
        assert not got[k][gone].any() and not torch.signbit(got[k][gone]).any()
    assert torch.equal(got[1][1], h0[1]) and torch.equal(got[4][1], dh[1])  # the empty sequence


def _strided(layout, batch, steps, ch, dt, fill):
    """Tensors of one layout: whether the halves of one buffer, time before batch, or apart
    from a base that is aligned to its element alone."""
    if layout == "halves":
        return fill(torch.empty(batch, steps, 2 * ch, dtype=dt, device="cuda"))
    if layout == "time first":
        return fill(torch.empty(steps, batch, 2 * ch, dtype=dt, device="cuda").transpose(0, 1))
    flat = torch.empty(1 + batch * (steps + 1) * (2 * ch + 3), dtype=dt, device="cuda")
    return fill(flat[1:].view(batch, steps + 1, 2 * ch + 3)[:, :steps, :2 * ch])


@pytest.mark.parametrize("dt", [F, B])
@pytest.mark.parametrize("ch", [64, 50, 33])
@pytest.mark.parametrize("layout", ["halves", "time first", "odd"])
def test_layouts(layout, ch, dt):
    batch, steps = 3, 150
    z, x, h0, dy, dh = _inputs(ch, batch, steps, ch, dt)
    plain = _run(z, x, h0, None, dy, dh)

    def fill(t):
        t[..., :ch], t[..., ch:] = z, x
        return t

    zx = _strided(layout, batch, steps, ch, dt, fill)
    dzx = _strided(layout, batch, steps, ch, dt, lambda t: t)
    dy2 = _strided(layout, batch, steps, ch, dt, lambda t: t)[..., :ch]
    dy2.copy_(dy)
    y = _strided(layout, batch, steps, ch, dt, lambda t: t)[..., ch:]
    got = _run(zx[..., :ch], zx[..., ch:], h0, None, dy2, dh, dzx[..., :ch], dzx[..., ch:], y)
    _check(got, z, x, h0, None, dy, dh)
    for g, p in zip(got, plain):  # the split of the steps does not depend on the layout
        assert torch.equal(g, p)


@pytest.mark.parametrize("dt", [F, B])
@pytest.mark.parametrize("batch,steps,ch", [(2, 150, 33), (3, 200, 57), (2, 129, 58), (2, 300, 61), (2, 700, 62),
                                            (1, 1100, 121), (2, 257, 123), (40, 140, 61), (3, 140, 1001)])
def test_rows_off_every_alignment(batch, steps, ch, dt):
    """Rows that begin at any element, among values that are not numbers and stay as they are."""
    z, x, h0, dy, dh = _inputs(ch + steps, batch, steps, ch, dt)

    def among(t, shift, gap):
        whole = torch.full((shift + batch * steps * (ch + gap) + 9,), float("nan"), dtype=dt, device="cuda")
        view = whole[shift:shift + batch * steps * (ch + gap)].view(batch, steps, ch + gap)[..., :ch]
        if t is not None:
            view.copy_(t)
        return whole, view

    for shift in range(0, 8, 3):
        ins = [among(t, shift + i, shift + 2 * i) for i, t in enumerate((z, x, dy))]
        outs = [among(None, shift + i, 1 + shift + i) for i in range(3)]
        (_, z2), (_, x2), (_, dy2) = ins
        _check(_run(z2, x2, h0, None, dy2, dh, *(v for _, v in outs)), z, x, h0, None, dy, dh)
        for whole, view in outs:
            assert not bool(view.isnan().any())
            view.fill_(float("nan"))
            assert bool(whole.isnan().all())


@pytest.mark.parametrize("dt", [F, B])
@pytest.mark.parametrize("batch,steps,ch", [(1, 2000, 5), (1, 3713, 33), (30, 1345, 1), (2, 1700, 130)])
def test_long_sequences_of_few_channels(batch, steps, ch, dt):
    """Ragged, with and without the kept states, and with the states replaced in place."""
    z, x, h0, dy, dh = _inputs(steps + ch, batch, steps, ch, dt)
    lengths = torch.tensor([steps - 700 * (b % 3) for b in range(batch)], dtype=torch.int32, device="cuda")
    got = _run(z, x, h0, lengths, dy, dh)
    ref, bound = recurrence(z, x, h0, lengths, dy, dh)
    for name, g, r, e in zip(("y", "h_last", "dz", "dx", "dh0"), got, ref, bound):
        assert_within(g, r, e, name)
    h = ac.adacomp_recurrence_init(ch, CODE[dt])
    y, dz, dx = (torch.full_like(z, -9.0) for _ in range(3))
    state, carry, grad = h0.clone(), _carry(h, batch, steps), dh.clone()
    ac.adacomp_recurrence_forward(h, z, x, y, h0=state, lengths=lengths, h_last=state)
    for g, r, e, name in zip((y, state), ref, bound, ("y without carry", "h_last in place")):
        assert_within(g, r, e, name)
    ac.adacomp_recurrence_forward(h, z, x, y, h0=h0, lengths=lengths, carry=carry)
    assert torch.equal(y, got[0])
    ac.adacomp_recurrence_backward(h, z, x, dy, carry, dz, dx, lengths=lengths, dh_last=grad, dh0=grad)
    for g, e in zip((dz, dx, grad), got[2:]):
        assert torch.equal(g, e)


def test_what_lies_between_the_rows_is_kept():
    batch, steps, ch = 2, 40, 21
    z, x, h0, dy, dh = _inputs(1, batch, steps, ch, B)
    outs = [torch.full((batch, steps + 2, ch + 5), -7.0, dtype=B, device="cuda") for _ in range(3)]
    views = [o[:, 1:steps + 1, 2:ch + 2] for o in outs]
    _run(z, x, h0, None, dy, dh, views[0], views[1], views[2])
    for o, v in zip(outs, views):
        assert not (v == -7.0).all()
        v.fill_(-7.0)
        assert bool((o == -7.0).all())


def test_optional_inputs_and_outputs():
    z, x, h0, dy, dh = _inputs(8, 2, 140, 48, F)
    full = _run(z, x, torch.zeros_like(h0), None, dy, torch.zeros_like(dh))
    h = ac.adacomp_recurrence_init(48, ac.F32)
    y, dz, dx = torch.empty_like(z), torch.empty_like(z), torch.empty_like(z)
    ac.adacomp_recurrence_forward(h, z, x, y)
    assert torch.equal(y, full[0])
    carry = _carry(h, 2, 140)
    state = h0.clone()
    ac.adacomp_recurrence_forward(h, z, x, y, h0=state, h_last=state, carry=carry)  # the state in place
    assert torch.equal(state, _run(z, x, h0, None, dy, dh)[1])
    ac.adacomp_recurrence_forward(h, z, x, y, carry=carry)
    ac.adacomp_recurrence_backward(h, z, x, dy, carry, dz, dx)
    assert torch.equal(dz, full[2]) and torch.equal(dx, full[3])
    grad = dh.clone()
    ac.adacomp_recurrence_backward(h, z, x, dy, carry, dz, dx, dh_last=grad, dh0=grad)
    ref = _run(z, x, torch.zeros_like(h0), None, dy, dh)
    assert torch.equal(grad, ref[4]) and torch.equal(dz, ref[2])


def test_no_steps_and_no_sequences():
    h = ac.adacomp_recurrence_init(10, ac.F32)
    empty = torch.empty(3, 0, 10, device="cuda")
    h0, last = torch.randn(3, 10, device="cuda"), torch.empty(3, 10, device="cuda")
    carry = torch.empty(0, device="cuda")
    ac.adacomp_recurrence_forward(h, empty, empty, empty, h0=h0, h_last=last, carry=carry)
    assert torch.equal(last, h0)
    ac.adacomp_recurrence_forward(h, empty, empty, empty, h_last=last)
    assert not last.any()
    ac.adacomp_recurrence_backward(h, empty, empty, empty, carry, empty, empty, dh_last=h0, dh0=last)
    assert torch.equal(last, h0)
    none = torch.empty(0, 5, 10, device="cuda")
    ac.adacomp_recurrence_forward(h, none, none, none)


def test_steps_one_by_one_carry_the_state():
    """Single-token calls that hand the state on, against the whole sequence at once."""
    batch, steps, ch = 4, 40, 96
    z, x, h0, _, _ = _inputs(6, batch, steps, ch, F)
    ref, bound = recurrence(z, x, h0)
    h = ac.adacomp_recurrence_init(ch, ac.F32)
    state, y = h0.clone(), torch.empty_like(z)
    for t in range(steps):
        ac.adacomp_recurrence_forward(h, z[:, t:t + 1], x[:, t:t + 1], y[:, t:t + 1], h0=state, h_last=state)
    assert_within(y, ref[0], bound[0], "y")
    assert_within(state, ref[1], bound[1], "state")


@pytest.mark.parametrize("dt", [F, B])
def test_closed_open_and_infinite_gates(dt):
    """Gates far out on both sides: a state that is kept for good, or forgotten at once."""
    batch, steps, ch = 2, 300, 40
    z, x, h0, dy, dh = _inputs(11, batch, steps, ch, dt)
    z[:, :, 0:8] = 80.0
    z[:, :, 8:16] = -80.0
    z[:, :, 16:20] = float("inf")
    z[:, :, 20:24] = -float("inf")
    z[:, ::3, 24:32] = 30.0
    _check(_run(z, x, h0, None, dy, dh), z.clamp(-1e3, 1e3), x, h0, None, dy, dh)


def test_non_finite_values_stay_in_their_channel_and_after_their_step():
    z, x, h0, dy, dh = _inputs(12, 2, 300, 70, F)
    clean = _run(z, x, h0, None, dy, dh)
    x[1, 137, 3] = float("nan")
    z[0, 200, 69] = float("nan")
    got = _run(z, x, h0, None, dy, dh)
    y = clean[0].clone()
    assert torch.isnan(got[0][1, 137:, 3]).all() and torch.isnan(got[0][0, 200:, 69]).all()
    ok = torch.ones_like(y, dtype=torch.bool)
    ok[1, 137:, 3] = False
    ok[0, 200:, 69] = False
    assert torch.isfinite(got[0][ok]).all()
    others = torch.ones(2, 300, 70, dtype=torch.bool, device="cuda")
    others[1, :, 3] = False
    others[0, :, 69] = False
    for k in (0, 2, 3):
        assert torch.equal(got[k][others], clean[k][others])


def test_gradients_against_differences():
    """Directional derivatives of the kernel's own forward pass in 32 bits; the bound is the
    central difference's (a third derivative of order one per element) and the rounding's."""
    batch, steps, ch = 2, 200, 33
    z, x, h0, dy, dh = _inputs(5, batch, steps, ch, F, gate=1.0)
    h = ac.adacomp_recurrence_init(ch, ac.F32)
    grads = _run(z, x, h0, None, dy, dh)[2:]
    gen, e = _gen(50), 2.0 ** -7

    def loss(z, x, h0):
        y, last = torch.empty_like(z), torch.empty_like(h0)
        ac.adacomp_recurrence_forward(h, z, x, y, h0=h0, h_last=last)
        return float((y.double() * dy.double()).sum() + (last.double() * dh.double()).sum())

    for k, grad in enumerate(grads):
        args = [z, x, h0]
        v = _rand(gen, *args[k].shape)
        ends = []
        for s in (e, -e):
            moved = list(args)
            moved[k] = args[k] + s * v
            ends.append(loss(*moved))
        got, want = (ends[0] - ends[1]) / (2 * e), float((grad.double() * v.double()).sum())
        scale = float((batch * steps * ch) ** 0.5)
        assert abs(got - want) <= scale * (4 * e * e + 64 * U / e), (k, got, want)


def test_offsets_past_32_bits():
    """Sequences 2^31 + 64 elements apart."""
    batch, steps, ch, gap = 2, 150, 40, 2 ** 31 + 64
    z, x, h0, dy, dh = _inputs(21, batch, steps, ch, B)
    flat = torch.empty(gap + steps * 2 * ch, dtype=B, device="cuda")
    zx = flat.as_strided((batch, steps, 2 * ch), (gap, 2 * ch, 1))
    zx[..., :ch], zx[..., ch:] = z, x
    out = torch.empty(gap + steps * 2 * ch, dtype=B, device="cuda").as_strided((batch, steps, 2 * ch), (gap, 2 * ch, 1))
    ref = _run(z, x, h0, None, dy, dh)
    got = _run(zx[..., :ch], zx[..., ch:], h0, None, dy, dh, out[..., :ch], out[..., ch:])
    assert all(torch.equal(a, r) for a, r in zip(got, ref))


def test_same_bits_on_another_stream_and_in_a_graph():
    z, x, h0, dy, dh = _inputs(31, 3, 1500, 200, B)
    ref = _run(z, x, h0, None, dy, dh)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            assert all(torch.equal(a, r) for a, r in zip(_run(z, x, h0, None, dy, dh), ref))
    side.synchronize()
    h = ac.adacomp_recurrence_init(200, ac.BF16)
    out = [torch.zeros_like(t) for t in ref]
    carry = _carry(h, 3, 1500)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ac.adacomp_recurrence_forward(h, z, x, out[0], h0=h0, h_last=out[1], carry=carry)
        ac.adacomp_recurrence_backward(h, z, x, dy, carry, out[2], out[3], dh_last=dh, dh0=out[4])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, r) for a, r in zip(out, ref))


@pytest.mark.parametrize("silent", [0, 1])
@pytest.mark.parametrize("dt,batch,steps,ch", [(F, 3, 1500, 200), (B, 3, 1500, 200), (F, 3, 1100, 301)])
def test_a_wait_within_a_cluster_that_runs_out(dt, batch, steps, ch, silent):
    """One CTA of every cluster writes nothing to the others: every wait ends at its timeout, in the
    first of several rounds, all results are NaN, and the next calls are as they were."""
    z, x, h0, dy, dh = _inputs(3, batch, steps, ch, dt)
    h = ac.adacomp_recurrence_init(ch, CODE[dt])
    carry, kept = _carry(h, batch, steps), _carry(h, batch, steps)

    def run(carry_in, carry_out):
        y, dz, dx = (torch.full_like(z, -9.0) for _ in range(3))
        last, dh0 = torch.zeros_like(h0), torch.zeros_like(h0)
        ac.adacomp_recurrence_forward(h, z, x, y, h0=h0, h_last=last, carry=carry_out)
        ac.adacomp_recurrence_backward(h, z, x, dy, carry_in, dz, dx, dh_last=dh, dh0=dh0)
        return y, last, dz, dx, dh0

    before = run(carry, carry)
    ac.adacomp_recurrence_set_timeout_ns(h, 20_000_000)  # 20 ms
    ac.adacomp_recurrence_set_fault_injection(h, silent)
    for t in run(carry, kept):
        assert bool(t.isnan().all())
    ac.adacomp_recurrence_set_fault_injection(h)
    for got, want in zip(run(carry, kept), before):
        assert torch.equal(got, want)
    assert torch.equal(kept, carry)


def _kind(t):
    """0 where finite, 1 and 2 where an infinity of either sign, 3 where not a number."""
    return torch.isposinf(t) + 2 * torch.isneginf(t) + 3 * torch.isnan(t)


@pytest.mark.parametrize("dt", [F, B])
@pytest.mark.parametrize("batch,steps,ch", [(3, 3, 50), (25, 14, 900), (3, 40, 70), (5, 200, 1000), (5, 200, 1001),
                                            (16, 150, 1024), (3, 1500, 200), (3, 1100, 301), (1, 2000, 37),
                                            (1, 4000, 64), (30, 1345, 9)])
def test_infinite_states_and_gradients_stay_infinite(batch, steps, ch, dt):
    """Infinities in h0, x, dh_last and dy, behind gates whose product over a chunk of steps vanishes
    in fp32 although none of them does: as by the definition, a state or gradient stays infinite,
    and only two infinities of unlike sign make a value that is not a number."""
    z, x, h0, dy, dh = _inputs(batch + steps, batch, steps, ch, dt)
    z.copy_((torch.rand(z.shape, generator=_gen(1), device="cuda") - 7.5).to(dt))
    inf, early, late = float("inf"), min(1, steps - 1), steps - 1 - (steps > 8)
    h0[:, 0], h0[:, 1], h0[:, 3], h0[0, 4] = inf, -inf, inf, -inf
    x[:, early, 2], x[:, late, 3], x[:, early, 4] = inf, -inf, -inf
    dh[:, 5], dh[:, 6], dh[:, 8] = inf, -inf, inf
    dy[:, late, 7], dy[:, early, 8] = -inf, -inf
    got = _run(z, x, h0, None, dy, dh)
    ref, bound = recurrence(z, x, h0, None, dy, dh)
    for name, g, r, e in zip(("y", "h_last", "dz", "dx", "dh0"), got, ref, bound):
        same = _kind(g) == _kind(r)
        assert bool(same.all()), (name, (~same).nonzero()[:3].tolist(), g[~same][:3], r[~same][:3])
        assert_within(g[..., 9:], r[..., 9:], e[..., 9:], name)
