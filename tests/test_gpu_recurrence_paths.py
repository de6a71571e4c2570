"""Every kernel of the recurrence over several of its turns, rounds and tiles, ragged and whole,
against the plain form in 64 bits (GPU); and that the sizes given here do reach the kernels that
they are for, so that a rule that is changed leaves none without a test."""
import re

import pytest
import torch

import residual_gradient_compression_gb300 as ac
from _gpu import ensure_built
from _train import assert_within, recurrence

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:DEBUG")]
F, B = torch.float32, torch.bfloat16
CODE = {F: ac.F32, B: ac.BF16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_built()


def kernels_of(call, path):
    """The kernels that a call launches, as file:kernel<template arguments>, from its graph."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        call()
    graph.debug_dump(str(path))
    names = []
    for unit, rest in re.findall(r"_\d+_(\w+?)_cu_[0-9a-f]{8}[_\d]+(rec_\w+?)Evv?N", path.read_text()):
        kernel, args = re.match(r"(rec_\w+?_kernel)I(.*)$", rest).groups()
        kind = "b" if args.startswith("13__nv_bfloat16") else "f"
        numbers = [n.replace("n", "-") for n in re.findall(r"L[ib](n?\d+)E", args)]
        names.append(f"{unit}:{kernel}<{','.join([kind] + numbers)}>")
    return names


def _tensor(batch, steps, ch, pad, dt, gen=None, offset=0.0):
    """[batch, steps, channels] in rows that are `pad` elements longer."""
    whole = torch.full((batch, steps, ch + pad), float("nan"), dtype=dt, device="cuda")
    view = whole[..., :ch]
    if gen is not None:
        view.copy_((torch.randn(batch, steps, ch, generator=gen, device="cuda") + offset).to(dt))
    return whole, view


# (type, batch, steps, channels, longer rows; kernels of the forward pass and of the backward pass). Two columns per
# lane: from 14592 columns on; one: from 4864 on; below that, clusters, or all chunks at once where there are many.
MANY = "recurrence:rec_forward_kernel<{}>", "recurrence:rec_backward_kernel<{}>"
FEW = "recurrence:rec_forward_few_kernel<{}>", "recurrence:rec_backward_few_kernel<{}>"
CLUSTER = "recurrence_split:rec_forward_kernel<{},0>", "recurrence_split:rec_backward_kernel<{},0>"


def _many(forward, backward):
    return [MANY[0].format(forward)], [MANY[1].format(backward)]


def _cluster(args):
    return [CLUSTER[0].format(args)], [CLUSTER[1].format(args)]


def _chunks(kind, by):
    return tuple([f"recurrence_split:rec_totals_kernel<{kind},{by},{back}>",
                  f"recurrence_split:rec_states_kernel<{kind},{back}>",
                  f"recurrence_split:rec_{'backward' if back else 'forward'}_kernel<{kind},{by},1>"] for back in (0, 1))


CASES = [
    # two columns per lane: several turns of eight warps, several kept states; channels that end inside a lane's pair
    (B, 16, 200, 1024, 0, *_many("b,16,2", "b,16,2")),
    (F, 16, 200, 1024, 0, *_many("f,16,2", "f,16,1")),
    (B, 15, 300, 1024, 0, *_many("b,16,2", "b,16,2")),
    (F, 15, 300, 1024, 0, *_many("f,16,2", "f,16,1")),
    (B, 15, 70, 1024, 0, *_many("b,16,2", "b,16,2")),
    (B, 16, 200, 1023, 1, *_many("b,16,2", "b,16,2")),
    (F, 16, 200, 1021, 3, *_many("f,16,2", "f,16,1")),
    # one column per lane; rows of any alignment by the 16 bytes that hold them, by pairs, and one by one
    (B, 5, 300, 1024, 0, *_many("b,16,1", "b,16,1")),
    (F, 5, 300, 1021, 3, *_many("f,16,1", "f,16,1")),
    (B, 5, 300, 1001, 0, *_many("b,-2,1", "b,-2,1")),
    (F, 5, 300, 1001, 0, *_many("f,-4,1", "f,-4,1")),
    (B, 16, 200, 1001, 0, *_many("b,-2,1", "b,-2,1")),
    (F, 16, 200, 1001, 0, *_many("f,-4,1", "f,-4,1")),
    (B, 5, 300, 1002, 0, *_many("b,4,1", "b,4,1")),
    (B, 160, 300, 33, 0, *_many("b,2,1", "b,2,1")),
    (F, 160, 300, 33, 0, *_many("f,4,1", "f,4,1")),
    # a thread per column
    (B, 25, 3, 900, 0, [FEW[0].format("b")], [FEW[1].format("b,4")]),
    (F, 25, 3, 900, 0, [FEW[0].format("f")], [FEW[1].format("f,4")]),
    (B, 25, 14, 900, 0, [FEW[0].format("b")], [FEW[1].format("b,16")]),
    (F, 25, 14, 900, 0, [FEW[0].format("f")], [FEW[1].format("f,16")]),
    (F, 25, 20, 900, 0, [FEW[0].format("f")], [FEW[1].format("f,32")]),
    (B, 25, 20, 900, 0, [FEW[0].format("b")], [MANY[1].format("b,4,1")]),
    # clusters of eight and of sixteen in six rounds (a barrier's phase comes round in the fifth)
    (F, 4, 3000, 400, 0, *_cluster("f,16")),
    (B, 4, 6000, 256, 0, *_cluster("b,16")),
    (F, 4, 3000, 401, 0, *_cluster("f,-4")),
    (B, 4, 6000, 227, 0, *_cluster("b,-2")),
    (F, 60, 3000, 24, 0, *_cluster("f,4")),
    (B, 60, 3000, 26, 0, *_cluster("b,4")),
    (B, 60, 3000, 25, 0, *_cluster("b,2")),
    # all chunks at once: aligned rows, a last chunk of one step, a last tile of a few columns; and channels numbered through
    (F, 1, 2000, 64, 0, *_chunks("f", 16)),
    (F, 1, 1700, 36, 0, *_chunks("f", 16)),
    (B, 1, 4000, 64, 0, *_chunks("b", 16)),
    (B, 1, 3713, 40, 0, *_chunks("b", 16)),
    (B, 1, 4000, 72, 0, *_chunks("b", 16)),
    (F, 1, 2000, 63, 0, *_chunks("f", -4)),
    (B, 1, 4000, 57, 0, *_chunks("b", -2)),
    (F, 3, 2000, 5, 0, *_chunks("f", 4)),
    (B, 3, 2000, 6, 0, *_chunks("b", 4)),
    (B, 3, 2000, 5, 0, *_chunks("b", 2)),
]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("dt,batch,steps,ch,pad,forward,backward", CASES,
                         ids=[f"{'f32' if c[0] is F else 'bf16'}-{c[1]}x{c[2]}x{c[3]}+{c[4]}" for c in CASES])
def test_against_64_bits(dt, batch, steps, ch, pad, forward, backward, ragged, tmp_path):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(batch + steps + ch + ragged)
    (_, z), (_, x), (_, dy) = (_tensor(batch, steps, ch, pad, dt, gen, o) for o in (2.0, 0.0, 0.0))
    (ys, y), (dzs, dz), (dxs, dx) = (_tensor(batch, steps, ch, pad, dt) for _ in range(3))
    h0, dh = torch.randn(batch, ch, generator=gen, device="cuda"), torch.randn(batch, ch, generator=gen, device="cuda")
    lengths = None
    if ragged:  # whole, empty, one step, and spread; NaN past them
        ends = ([steps, 0, 1] if batch > 2 else []) + [steps - 1 - (b * 97) % steps for b in range(batch)]
        lengths = torch.tensor(ends[:batch], dtype=torch.int32, device="cuda")
        gone = torch.arange(steps, device="cuda")[None, :] >= lengths[:, None]
        for t in (z, x, dy):
            t[gone] = float("nan")
    h = ac.adacomp_recurrence_init(ch, CODE[dt])
    last, dh0 = torch.empty_like(h0), torch.empty_like(h0)
    carry = torch.full((ac.adacomp_recurrence_carry_bytes(h, batch, steps) // 4,), float("nan"), device="cuda")

    def run_forward():
        ac.adacomp_recurrence_forward(h, z, x, y, h0=h0, lengths=lengths, h_last=last, carry=carry)

    def run_backward():
        ac.adacomp_recurrence_backward(h, z, x, dy, carry, dz, dx, lengths=lengths, dh_last=dh, dh0=dh0)

    run_forward()
    run_backward()
    ref, bound = recurrence(z, x, h0, lengths, dy, dh)
    got = dict(y=y, h_last=last, dz=dz, dx=dx, dh0=dh0)
    for (name, g), r, e in zip(got.items(), ref, bound):
        assert_within(g, r, e, name)
    for whole in (ys, dzs, dxs):  # what lies between the rows
        assert bool(whole[..., ch:].isnan().all())
    again = torch.empty_like(y)  # and without the kept states
    ac.adacomp_recurrence_forward(h, z, x, again, h0=h0, lengths=lengths)
    assert_within(again, ref[0], bound[0], "y without kept states")
    assert kernels_of(run_forward, tmp_path / "forward.dot") == forward
    assert kernels_of(run_backward, tmp_path / "backward.dot") == backward


def test_every_kernel_is_reached():
    """The instances that the rules can choose are those of the cases."""
    seen = {k for c in CASES for k in c[5] + c[6]}
    want = {MANY[0].format(a) for a in ("b,16,2", "f,16,2", "b,16,1", "f,16,1", "b,-2,1", "f,-4,1", "b,4,1", "b,2,1", "f,4,1")}
    want |= {MANY[1].format(a) for a in ("b,16,2", "b,16,1", "f,16,1", "b,-2,1", "f,-4,1", "b,4,1", "b,2,1", "f,4,1")}
    want |= {FEW[0].format(a) for a in "bf"} | {FEW[1].format(a) for a in ("b,4", "f,4", "b,16", "f,16", "f,32")}
    for a in ("f,16", "b,16", "f,-4", "b,-2", "f,4", "b,4", "b,2"):
        want |= {k.format(a) for k in CLUSTER}
        for part in _chunks(*a.split(",")):
            want |= set(part)
    assert seen == want
