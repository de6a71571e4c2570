"""The gradient norm and the AdamW step (GPU): bit for bit against the same fp32 operations
in torch, as the header defines them, and against the formulas in 64 bits with rounding
bounds."""
import math

import numpy as np
import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built, workspace
from _train import U, assert_within, blocks, to_e4m3

pytestmark = pytest.mark.gpu
F, B = torch.float32, torch.bfloat16
CODE = {F: ac.F32, B: ac.BF16}
LR, BETA1, BETA2, EPS = 1e-3, 0.9, 0.999, 1e-8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _corrections(t):
    return float(np.float32(1 - BETA1 ** t)), float(np.float32(1 - BETA2 ** t))


class Net:
    """Weights, gradients and states of several tensors, and copies to compare with."""

    def __init__(self, sizes, wts, gts, bits, seed=0, decay=None, fresh=False, copies=False):
        gen = _gen(seed)
        rand = lambda n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
        self.sizes, self.bits = sizes, bits
        self.decay = [0.01 * (i % 3) for i in range(len(sizes))] if decay is None else decay
        self.h = ac.adacomp_adamw_init(sizes, [CODE[t] for t in wts], [CODE[t] for t in gts], self.decay, bits)
        self.w = [(0.02 * rand(n)).to(t) for n, t in zip(sizes, wts)]
        self.g = [(1e-3 * rand(n)).to(t) for n, t in zip(sizes, gts)]
        self.copies = [torch.zeros(n, dtype=B, device="cuda") for n in sizes] if copies else None
        zero = 0.0 if fresh else 1.0
        m = [zero * 2e-4 * rand(n) for n in sizes]
        u = [zero * (1e-3 * rand(n)).abs() for n in sizes]
        if bits == 8:
            self.m, self.ms = zip(*[self.encode(t, False) for t in m])
            self.v, self.vs = zip(*[self.encode(t, True) for t in u])
        else:
            self.m, self.v, self.ms, self.vs = m, [t * t for t in u], None, None

    @staticmethod
    def encode(v, positive):
        """fp32 values as e4m3 and a scale per block, each operation as the header states it."""
        r = blocks(v)
        top = r.abs().amax(1, keepdim=True)
        some = ~(top < 2.0 ** -96)
        most = torch.full_like(top, 448.0)  # a tensor: torch divides by, or into, a number through a reciprocal
        scale = torch.where(some, top / most, torch.zeros_like(top))
        code = (r * torch.where(some, most / top, torch.zeros_like(top))).to(torch.float8_e4m3fn)
        if positive:
            raw = code.view(torch.uint8)
            raw = torch.where((r > 0) & (raw == 0), torch.ones_like(raw), raw)
            code = raw.view(torch.float8_e4m3fn)
        return code.view(torch.uint8).view(-1)[:v.numel()].clone().view(torch.float8_e4m3fn), scale.view(-1)

    @staticmethod
    def decode(code, scale):
        return (blocks(code.float()) * scale[:, None]).view(-1)[:code.numel()]

    def state(self):
        parts = [self.w, self.m, self.v] + ([self.ms, self.vs] if self.bits == 8 else []) + \
            ([self.copies] if self.copies else [])
        return [t for part in parts for t in part]

    def step(self, t=3, scale=1.0, coefficient=None, lr=LR, stream=None):
        ac.adacomp_adamw_step(self.h, self.w, self.g, self.m, self.v, lr, BETA1, BETA2, EPS, *_corrections(t),
                              m_scale=self.ms, v_scale=self.vs, copies=self.copies, grad_scale=scale,
                              coefficient=coefficient, stream=stream)

    def expected(self, t=3, c=1.0, lr=LR):
        """What the step leaves, in the header's fp32 operations."""
        f = np.float32
        c1, c2 = _corrections(t)
        one = f(1.0)
        step, root = float(f(float(f(lr)) / c1)), float(f(1.0 / math.sqrt(c2)))
        b1, b2, r1, r2 = float(f(BETA1)), float(f(BETA2)), float(one - f(BETA1)), float(one - f(BETA2))
        ws, msn, vsn, mss, vss, cp = [], [], [], [], [], []
        for i in range(len(self.sizes)):
            kept = float(f(1.0 - float(f(lr)) * float(f(self.decay[i]))))
            if self.bits == 8:
                m = self.decode(self.m[i], self.ms[i])
                u = self.decode(self.v[i], self.vs[i])
                v = u * u
            else:
                m, v = self.m[i], self.v[i]
            g = self.g[i].float() * float(f(c))
            m = m * b1 + g * r1
            v = v * b2 + (g * g) * r2
            u = torch.sqrt(v)
            w = self.w[i].float() * kept - (m / (u * root + float(f(EPS)))) * step
            ws.append(w.to(self.w[i].dtype))
            cp.append(w.to(B))
            if self.bits == 8:
                m, s = self.encode(m, False)
                v, s2 = self.encode(u, True)
                mss.append(s)
                vss.append(s2)
            msn.append(m)
            vsn.append(v)
        return ws + msn + vsn + mss + vss + (cp if self.copies else [])


def _same(got, ref, what=""):
    assert len(got) == len(ref)
    for i, (a, r) in enumerate(zip(got, ref)):
        bytes_of = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
        assert a.dtype == r.dtype and torch.equal(bytes_of(a), bytes_of(r)), f"{what} buffer {i}: " + str(
            (a.float() != r.float()).nonzero()[:3].flatten().tolist())


SIZES = [1, 2, 3, 4, 7, 8, 31, 33, 127, 128, 129, 255, 256, 257, 511, 512, 1000, 2047, 2048, 2049, 4099, 8191, 8193,
         70_001, 1 << 20]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("wt,gt", [(F, F), (F, B), (B, F), (B, B)])
def test_step_is_the_headers_operations_bit_for_bit(wt, gt, bits):
    net = Net(SIZES, [wt] * len(SIZES), [gt] * len(SIZES), bits, seed=bits, copies=True)
    for t in (3, 4):
        ref = net.expected(t)
        net.step(t)
        _same(net.state(), ref, f"step {t}")


@pytest.mark.parametrize("bits", [32, 8])
def test_first_steps_from_zero_states_and_mixed_types(bits):
    wts = [F, B, F, B, B, F] * 4
    gts = [F, F, B, B, F, B] * 4
    net = Net([100 + 37 * i for i in range(24)], wts, gts, bits, fresh=True)
    for t in (1, 2, 3):
        ref = net.expected(t, c=0.25)
        net.step(t, scale=0.25)
        _same(net.state(), ref, f"step {t}")


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch_holds(bits):
    sizes = [1 + (i * 7919) % 3000 for i in range(1500)]
    net = Net(sizes, [F] * 1500, [B] * 1500, bits)
    ref = net.expected()
    net.step()
    _same(net.state(), ref)


@pytest.mark.parametrize("bits", [32, 8])
def test_against_64_bits(bits):
    net = Net([5000, 300], [F, F], [F, F], bits, seed=4)
    m = [t.double() if bits == 32 else Net.decode(t, s).double() for t, s in zip(net.m, net.ms or net.m)]
    v = [t.double() if bits == 32 else Net.decode(t, s).double() ** 2 for t, s in zip(net.v, net.vs or net.v)]
    w = [t.double() for t in net.w]
    t = 3
    net.step(t)
    f = np.float32
    b1, b2 = float(f(BETA1)), float(f(BETA2))
    c1, c2 = _corrections(t)
    for i in range(2):
        g = net.g[i].double()
        m2 = b1 * m[i] + (1 - b1) * g
        v2 = b2 * v[i] + (1 - b2) * g * g
        u2 = torch.sqrt(v2)
        q = (m2 / c1) / (u2 / math.sqrt(c2) + float(f(EPS)))
        ref = w[i] * (1 - float(f(LR)) * float(f(net.decay[i]))) - float(f(LR)) * q
        # each moment is a sum of two products; 1 - beta, of two fp32 numbers, is exact
        e_m = 4 * U * (b1 * m[i].abs() + (1 - b1) * g.abs())
        e_v = 5 * U * v2
        e_q = q.abs() * 9 * U + e_m / c1 / (u2 / math.sqrt(c2) + float(f(EPS)))
        e_w = 3 * U * (w[i].abs() + ref.abs()) + float(f(LR)) * (e_q + 3 * U * q.abs())
        assert_within(net.w[i], ref, e_w, f"w {i}")
        if bits == 32:
            assert_within(net.m[i], m2, e_m, f"m {i}")
            assert_within(net.v[i], v2, e_v, f"v {i}")
            continue
        for code, scale, value, e in ((net.m[i], net.ms[i], m2, e_m), (net.v[i], net.vs[i], u2, 4 * U * u2)):
            rows = blocks(value)
            top = rows.abs().amax(1, keepdim=True)
            assert_within(scale, top[:, 0] / 448, 8 * U * top[:, 0] / 448, "scale")
            # half a step of e4m3 (2^-4 of the value, or half of the smallest), and 2^-9 where u is kept from 0
            back = blocks(code.double())
            near = rows * 448 / top
            slack = near.abs() * 2.0 ** -4 + 2.0 ** -9 + 448 * blocks(e) / top
            assert_within(back, near, slack, "code")
            off = (back != to_e4m3(near)) & (back != 2.0 ** -9)
            assert float(off.float().mean()) < 1e-3  # but for ties that rounding moves, the nearest number


@pytest.mark.parametrize("exponent", [0, -31, 29, -59])
def test_root_and_quotient_round_correctly_for_every_significand(exponent):
    """beta2 = 0.5 and no gradient: v = 2^exponent * [1, 4), all 2^24 values; lr * weight_decay
    = 1 and w = 0 leave w = -m / (u + eps), whose rounding torch's root and quotient give."""
    n = 1 << 24
    h = ac.adacomp_adamw_init([n], [ac.F32], [ac.F32], [1.0], 32)
    v = (torch.arange(n, dtype=torch.int32, device="cuda") + ((127 + exponent) << 23)).view(F)
    want_v = v.clone()
    v *= 2.0
    gen = _gen(exponent + 100)
    m = torch.randn(n, generator=gen, device="cuda") * torch.exp2(
        torch.randint(-55, 55, (n,), generator=gen, device="cuda").float())
    m[::1001] = 0.0
    m[1::1003] = -0.0
    w, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    want = -((m * 0.5) / (torch.sqrt(want_v) + 2.0 ** -40))
    ac.adacomp_adamw_step(h, [w], [g], [m], [v], 1.0, 0.5, 0.5, 2.0 ** -40, 1.0, 1.0)
    assert torch.equal(v, want_v)
    assert torch.equal(w, want)


@pytest.mark.parametrize("bits", [32, 8])
def test_values_outside_the_usual_range(bits):
    """Moments and constants from one end of fp32 to the other, elements of both kinds in one lane."""
    n = 1 << 16
    net = Net([n], [F], [F], bits, seed=5)
    gen = _gen(77)
    net.g[0].copy_(torch.randn(n, generator=gen, device="cuda") * torch.exp2(
        torch.randint(-70, 62, (n,), generator=gen, device="cuda").float()))
    net.g[0][::5] = 0.0
    if bits == 32:
        net.m[0].copy_(torch.randn(n, generator=gen, device="cuda") * torch.exp2(
            torch.randint(-148, 100, (n,), generator=gen, device="cuda").float()))
        net.v[0].copy_(torch.rand(n, generator=gen, device="cuda") * torch.exp2(
            torch.randint(-148, 126, (n,), generator=gen, device="cuda").float()))
        net.v[0][::7] = 0.0
    for t in (1, 2, 1000):
        ref = net.expected(t)
        net.step(t)
        _same(net.state(), ref, f"step {t}")


def test_eight_bit_blocks_of_zeros_tiny_huge_and_few_values():
    n = 256 * 8 + 5
    net = Net([n], [F], [F], 8, fresh=True)
    g = net.g[0]
    g[0:256] = 0.0
    g[256:512] = 1e-36
    g[512:768] *= 1e20       # the squares overflow nothing yet
    g[768:1024] = 0.0
    g[770] = 5.0             # one value in a block of zeros
    g[1024:1280] = 1e-3
    g[1025] = 1e5            # the others' roots would round to zero
    for t in (1, 2):
        ref = net.expected(t)
        net.step(t)
        _same(net.state(), ref, f"step {t}")
    v = net.v[0].float()
    assert not v[:256].any() and (v[1024:1280] > 0).all() and torch.isfinite(net.w[0]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_not_finite_gradient_reaches_its_element_or_block_only(bits):
    net = Net([3000], [F], [F], bits)
    clean = Net([3000], [F], [F], bits)
    net.g[0][700] = float("nan")
    net.g[0][2000] = float("inf")
    net.step()
    clean.step()
    bad = (net.w[0] != clean.w[0]).nonzero().flatten().tolist()
    assert set(bad) <= {700, 2000} and math.isnan(net.w[0][700])
    same = [(a.float() == b.float()) for a, b in zip(net.m, clean.m)][0]
    where = set((~same).nonzero().flatten().tolist())
    assert where <= ({700, 2000} if bits == 32 else set(range(512, 768)) | set(range(1792, 2048)))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_coefficient_that_is_not_finite_leaves_everything(bits):
    net = Net([5000, 77], [F, B], [F, F], bits, copies=True)
    before = [t.clone() for t in net.state()]
    for bad in (float("nan"), float("inf")):
        net.step(coefficient=torch.tensor([bad], device="cuda"))
        _same(net.state(), before)
    ref = net.expected(c=0.5)
    net.step(coefficient=torch.tensor([0.5], device="cuda"), scale=float("nan"))
    _same(net.state(), ref)


def test_copies_may_be_missing():
    net = Net([500, 600], [F, F], [F, F], 32, copies=True)
    ref = net.expected()
    first, net.copies = net.copies, [net.copies[0], None]
    net.step()
    net.copies = first
    _same(net.state()[:-1], ref[:-1])
    assert not first[1].any()


def test_nothing_past_a_tensors_end_is_touched():
    sizes = [1, 5, 255, 2049]
    net = Net(sizes, [B] * 4, [F] * 4, 8)
    wide = []
    for name in ("w", "m", "v"):
        new = []
        for t in getattr(net, name):
            raw = torch.full((t.numel() * t.element_size() + 512,), 0x5a, dtype=torch.uint8, device="cuda")
            inner = raw[:t.numel() * t.element_size()].view(t.dtype)
            inner.copy_(t)
            wide.append((raw, t.numel() * t.element_size()))
            new.append(inner)
        setattr(net, name, new)
    ref = net.expected()
    net.step()
    _same(net.state(), ref)
    for raw, end in wide:
        assert bool((raw[end:] == 0x5a).all())


def _norm(net, max_norm=0.0, scale=1.0, ws=None):
    ws = workspace(net.h.norm_ws_bytes) if ws is None else ws
    out = torch.empty(2, device="cuda")
    ac.adacomp_grad_norm(net.h, net.g, out, ws, max_norm=max_norm, grad_scale=scale)
    return [float(v) for v in out]


def _exact_norm(net):
    return math.sqrt(sum(float((g.double() ** 2).sum()) for g in net.g))


#: fp32 sums of at most 64 squares, each sum's relative error halved by the root, one final rounding
NORM_TOL = (64 + 2) * U / 2 + U


@pytest.mark.parametrize("sizes", [[1], [5, 3, 1], SIZES, [3_000_000], [1 + (i * 7919) % 3000 for i in range(3000)]])
@pytest.mark.parametrize("gt", [F, B, None])
def test_norm_and_clipping(sizes, gt):
    gts = [gt or (F if i % 2 else B) for i in range(len(sizes))]
    net = Net(sizes, [F] * len(sizes), gts, 32)
    ws = workspace(net.h.norm_ws_bytes)
    want = _exact_norm(net)
    for scale in (1.0, 0.125):
        n = scale * want
        for max_norm in (0.0, n / 3, 10 * n):
            norm, c = _norm(net, max_norm, scale, ws)
            assert abs(norm - n) <= NORM_TOL * n
            k = 1.0 if max_norm == 0 else min(1.0, max_norm / (n + 1e-6))
            assert abs(c - scale * k) <= (NORM_TOL + 4 * U) * scale * k
    assert _norm(net, 1.0, 1.0, ws) == _norm(net, 1.0, 1.0, ws)


@pytest.mark.parametrize("gt", [F, B])
def test_norm_of_values_whose_squares_overflow_or_vanish(gt):
    for factor in (1e25, 1e-24, 1e-35):
        net = Net([10_000, 77, 5], [F] * 3, [gt] * 3, 32)
        for g in net.g:
            g.mul_(1e3 * factor)
            g[3:5] = 0.0
        net.g[1].zero_()
        want = _exact_norm(net)
        norm, _ = _norm(net)
        assert abs(norm - want) <= NORM_TOL * want, (factor, norm, want)
    net.g[0].fill_(2.0 ** 60)
    net.g[2].fill_(2.0 ** -60)
    assert abs(_norm(net)[0] - 100 * 2.0 ** 60) <= NORM_TOL * 100 * 2.0 ** 60


def test_norm_of_zeros_infinities_and_nan():
    net = Net([4000, 9], [F, F], [F, B], 32)
    for g in net.g:
        g.zero_()
    assert _norm(net, 1.0) == [0.0, 1.0]
    for bad in (float("inf"), float("nan")):
        net.g[1][8] = bad
        norm, c = _norm(net, 1.0)
        assert not math.isfinite(norm) and math.isnan(c)
        net.g[1][8] = 0.0
    net.g[0].fill_(3e38)  # a norm past fp32's range
    assert _norm(net)[0] == math.inf


def test_norm_and_step_in_a_graph_and_on_another_stream():
    sizes = [300_000, 5000, 33]
    nets = [Net(sizes, [F] * 3, [B] * 3, 8, seed=7) for _ in range(3)]
    rs = [torch.empty(2, device="cuda") for _ in nets]
    wss = [workspace(n.h.norm_ws_bytes) for n in nets]

    def both(i, stream=None):
        ac.adacomp_grad_norm(nets[i].h, nets[i].g, rs[i], wss[i], max_norm=0.1, stream=stream)
        nets[i].step(coefficient=rs[i][1:], stream=stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        graph.replay()
        both(1)
        both(2, side)
    torch.cuda.synchronize()
    for i in (0, 2):
        _same(nets[i].state(), nets[1].state())
        assert torch.equal(rs[i], rs[1])


def test_a_tensor_past_2_to_31_elements():
    n, tail = 2 ** 31 + 777, 5000
    h = ac.adacomp_adamw_init([n], [ac.BF16], [ac.BF16], [0.01], 8)
    w, g = torch.zeros(n, dtype=B, device="cuda"), torch.zeros(n, dtype=B, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    nb = -(-n // 256)
    ms, vs = torch.zeros(nb, device="cuda"), torch.zeros(nb, device="cuda")
    first = n - tail - (n - tail) % 256  # a block's start: the tail is a tensor of its own
    small = Net([n - first], [B], [B], 8, seed=3, fresh=True, decay=[0.01])
    w[first:], g[first:] = small.w[0], small.g[0]
    ac.adacomp_adamw_step(h, [w], [g], [m], [v], LR, BETA1, BETA2, EPS, *_corrections(3), m_scale=[ms], v_scale=[vs])
    small.step(3)
    _same([w[first:], m.view(torch.uint8)[first:].view(torch.float8_e4m3fn),
           v.view(torch.uint8)[first:].view(torch.float8_e4m3fn), ms[first // 256:], vs[first // 256:]], small.state())
    assert not w[:first].any()
    out, ws = torch.empty(2, device="cuda"), workspace(h.norm_ws_bytes)
    ac.adacomp_grad_norm(h, [g], out, ws)
    want = _exact_norm(small)
    assert abs(float(out[0]) - want) <= NORM_TOL * want
