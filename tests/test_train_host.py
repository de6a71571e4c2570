"""Host-side checks of the training operators' entry points (no GPU): argument errors come
back before any launch, and sizes are as the header states."""
import ctypes
import os
import re

import pytest
import torch

import residual_gradient_compression_gb300 as ac
from residual_gradient_compression_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # a 16-byte-aligned stand-in address; no call below reaches the GPU


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    ac.lib()


def _status(call, *args):
    with pytest.raises(ac.AdacompError) as e:
        call(*args)
    return e.value.status


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "adacomp.h")).read()
    for name, value in (("ADACOMP_RECURRENCE_CHUNK", ac.RECURRENCE_CHUNK), ("ADACOMP_ADAMW_BLOCK", ac.ADAMW_BLOCK)):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == value


@pytest.mark.parametrize("dim,xd,wd,eps", [(0, 0, 0, 1e-5), (-1, 0, 0, 1e-5), (8, 2, 0, 1e-5), (8, 0, -1, 1e-5),
                                           (8, 0, 0, -1e-5), (8, 0, 0, float("nan")), (8, 0, 0, float("inf")),
                                           (2 ** 40, 0, 0, 1e-5)])
def test_layer_norm_init_refuses(dim, xd, wd, eps):
    p = ctypes.c_void_p(5)
    assert ac.lib().adacomp_layer_norm_init(ctypes.byref(p), dim, xd, wd, eps) == ac.ERR_INVALID_ARG
    assert p.value is None


def test_layer_norm_calls_refuse_before_launch():
    h = ac.adacomp_layer_norm_init(10, ac.BF16, ac.F32)
    L = ac.lib()
    good = [h.ptr, 4, A, 10, A, A, A, 10, A, A, None]

    def forward(**change):
        args = list(good)
        for k, v in change.items():
            args[int(k[1:])] = v
        return L.adacomp_layer_norm_forward(*args)

    for change in ({"a0": None}, {"a1": -1}, {"a1": 2 ** 31}, {"a2": None}, {"a3": -1}, {"a4": None}, {"a6": None},
                   {"a7": 9}):
        assert forward(**change) == ac.ERR_INVALID_ARG, change
    for change in ({"a2": A + 1}, {"a4": A + 2}, {"a5": A + 2}, {"a6": A + 1}, {"a8": A + 2}, {"a9": A + 1}):
        assert forward(**change) == ac.ERR_ALIGNMENT, change
    assert forward(a1=0, a2=None, a6=None) == ac.OK  # no rows: nothing to do

    need = ac.adacomp_layer_norm_backward_ws_bytes(h, 4)
    assert need > 0
    good = [h.ptr, 4, A, 10, A, 10, A, A, A, A, 10, A, A, A, need, None]

    def backward(**change):
        args = list(good)
        for k, v in change.items():
            args[int(k[1:])] = v
        return L.adacomp_layer_norm_backward(*args)

    for change in ({"a0": None}, {"a1": -1}, {"a2": None}, {"a3": -1}, {"a4": None}, {"a6": None}, {"a7": None},
                   {"a8": None}, {"a9": None}, {"a10": 9}, {"a11": None}, {"a13": None}):
        assert backward(**change) == ac.ERR_INVALID_ARG, change
    for change in ({"a2": A + 1}, {"a4": A + 1}, {"a6": A + 2}, {"a9": A + 1}, {"a11": A + 2}, {"a12": A + 2},
                   {"a13": A + 8}):
        assert backward(**change) == ac.ERR_ALIGNMENT, change
    assert backward(a14=need - 1) == ac.ERR_WORKSPACE


@pytest.mark.parametrize("ch,dt", [(0, 0), (-4, 0), (8, 2), (2 ** 40, 0)])
def test_recurrence_init_refuses(ch, dt):
    p = ctypes.c_void_p(5)
    assert ac.lib().adacomp_recurrence_init(ctypes.byref(p), ch, dt) == ac.ERR_INVALID_ARG
    assert p.value is None


def test_recurrence_calls_refuse_before_launch():
    h = ac.adacomp_recurrence_init(6, ac.F32)
    L = ac.lib()
    assert ac.adacomp_recurrence_carry_bytes(h, 3, 0) == 0
    assert ac.adacomp_recurrence_carry_bytes(h, 3, 129) == 3 * 3 * 6 * 4
    good = [h.ptr, 2, 5, A, 30, 6, A, 30, 6, A, A, A, 30, 6, A, A, None]

    def forward(**change):
        args = list(good)
        for k, v in change.items():
            args[int(k[1:])] = v
        return L.adacomp_recurrence_forward(*args)

    for change in ({"a0": None}, {"a1": -1}, {"a2": -1}, {"a1": 2 ** 31}, {"a3": None}, {"a6": None}, {"a11": None},
                   {"a4": -1}, {"a8": -6}, {"a13": 5}, {"a12": 5}):
        assert forward(**change) == ac.ERR_INVALID_ARG, change
    for change in ({"a3": A + 2}, {"a6": A + 1}, {"a9": A + 2}, {"a10": A + 2}, {"a11": A + 2}, {"a14": A + 2},
                   {"a15": A + 2}):
        assert forward(**change) == ac.ERR_ALIGNMENT, change
    assert forward(a1=0) == ac.OK
    good = [h.ptr, 2, 5, A, 30, 6, A, 30, 6, A, 30, 6, A, A, A, A, 30, 6, A, 30, 6, A, None]

    def backward(**change):
        args = list(good)
        for k, v in change.items():
            args[int(k[1:])] = v
        return L.adacomp_recurrence_backward(*args)

    for change in ({"a0": None}, {"a1": -1}, {"a2": 2 ** 31}, {"a3": None}, {"a6": None}, {"a9": None}, {"a12": None},
                   {"a15": None}, {"a18": None}, {"a17": 5}, {"a19": 5}):
        assert backward(**change) == ac.ERR_INVALID_ARG, change
    for change in ({"a3": A + 2}, {"a9": A + 2}, {"a12": A + 2}, {"a13": A + 2}, {"a14": A + 2}, {"a15": A + 2},
                   {"a18": A + 2}, {"a21": A + 2}):
        assert backward(**change) == ac.ERR_ALIGNMENT, change


def test_adamw_init_refuses():
    ok = ([5, 6], [0, 1], [1, 0])
    ac.adacomp_adamw_init(*ok)
    for bad in (([], [], []), ([0, 6], *ok[1:]), ([5, -6], *ok[1:]), ([5, 2 ** 41], *ok[1:]), ([1] * 65537,) * 3):
        types = [[0] * len(bad[0])] * 2
        assert _status(ac.adacomp_adamw_init, bad[0], *types) == ac.ERR_INVALID_ARG
    L, p = ac.lib(), ctypes.c_void_p(5)
    n, t = (ctypes.c_int64 * 2)(5, 6), (ctypes.c_int32 * 2)(0, 2)
    good = (ctypes.c_int32 * 2)(0, 1)
    for args in ((2, None, good, good, None, 32), (2, n, None, good, None, 32), (2, n, good, None, None, 32),
                 (2, n, t, good, None, 32), (2, n, good, t, None, 8), (2, n, good, good, None, 16),
                 (2, n, good, good, (ctypes.c_float * 2)(0.0, float("nan")), 32)):
        assert L.adacomp_adamw_init(ctypes.byref(p), *args, None) == ac.ERR_INVALID_ARG, args
        assert p.value is None
    with pytest.raises(ValueError):
        ac.adacomp_adamw_init([5, 6], [0], [0, 0])
    with pytest.raises(ValueError):
        ac.adacomp_adamw_init([5, 6], [0, 0], [0, 0], [0.1])


def _ptrs(*values):
    return (ctypes.c_void_p * len(values))(*values)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_step_refuses_before_launch(bits):
    h = ac.adacomp_adamw_init([300, 7], [0, 0], [0, 1], None, bits)
    one = _ptrs(A, A)
    scales = one if bits == 8 else None
    good = [h.ptr, one, one, one, one, scales, scales, None, 1e-3, 0.9, 0.999, 1e-8, 0.1, 0.001, 1.0, None, None]

    def step(**change):
        args = list(good)
        for k, v in change.items():
            args[int(k[1:])] = v
        return ac.lib().adacomp_adamw_step(*args)

    nan = float("nan")
    for change in ({"a0": None}, {"a1": None}, {"a2": None}, {"a3": None}, {"a4": None}, {"a1": _ptrs(A, None)},
                   {"a4": _ptrs(None, A)}, {"a5": None if bits == 8 else one}, {"a6": None if bits == 8 else one},
                   {"a8": nan}, {"a9": 1.0}, {"a9": -0.1}, {"a10": 1.0}, {"a10": nan}, {"a11": 0.0}, {"a11": nan},
                   {"a12": 0.0}, {"a13": 0.0}, {"a13": nan}):
        assert step(**change) == ac.ERR_INVALID_ARG, change
    for change in ({"a1": _ptrs(A, A + 8)}, {"a2": _ptrs(A + 4, A)}, {"a3": _ptrs(A + 2, A)}, {"a4": _ptrs(A, A + 1)},
                   {"a7": _ptrs(A + 2, None)}, {"a15": A + 2}):
        assert step(**change) == ac.ERR_ALIGNMENT, change


def test_grad_norm_refuses_before_launch():
    h = ac.adacomp_adamw_init([300, 7], [0, 0], [0, 1])
    one = _ptrs(A, A)
    good = [h.ptr, one, 1.0, 0.0, A, A, h.norm_ws_bytes, None]

    def norm(**change):
        args = list(good)
        for k, v in change.items():
            args[int(k[1:])] = v
        return ac.lib().adacomp_grad_norm(*args)

    for change in ({"a0": None}, {"a1": None}, {"a1": _ptrs(None, A)}, {"a2": 0.0}, {"a2": -1.0},
                   {"a2": float("inf")}, {"a3": float("nan")}, {"a4": None}, {"a5": None}):
        assert norm(**change) == ac.ERR_INVALID_ARG, change
    for change in ({"a1": _ptrs(A, A + 4)}, {"a4": A + 2}, {"a5": A + 8}):
        assert norm(**change) == ac.ERR_ALIGNMENT, change
    assert norm(a6=h.norm_ws_bytes - 1) == ac.ERR_WORKSPACE


def test_the_binding_refuses_tensors_that_do_not_fit():
    h = ac.adacomp_layer_norm_init(10, ac.F32, ac.F32)
    host = torch.zeros(4, 10)
    for x in (host, host.to(torch.bfloat16), torch.zeros(4, 11)):
        with pytest.raises(ValueError):
            ac.adacomp_layer_norm_forward(h, x, host[0], None, host)
    r = ac.adacomp_recurrence_init(10, ac.F32)
    with pytest.raises(ValueError):
        ac.adacomp_recurrence_forward(r, host, host, host)
    with pytest.raises(ValueError):
        ac.adacomp_recurrence_forward(r, host[None], host[None], host[None])
    with pytest.raises(ValueError):
        ac.adacomp_pointers([host])


def test_free_takes_null_and_twice():
    for name in ("layer_norm", "recurrence", "adamw"):
        getattr(ac.lib(), f"adacomp_{name}_free")(None)
    h = ac.adacomp_recurrence_init(10, ac.F32)
    ac.adacomp_recurrence_free(h)
    ac.adacomp_recurrence_free(h)


def test_recurrence_settings_refuse():
    L, h = ac.lib(), ac.adacomp_recurrence_init(10, ac.F32)
    assert L.adacomp_recurrence_set_timeout_ns(None, 5) == ac.ERR_INVALID_ARG
    assert L.adacomp_recurrence_set_fault_injection(None, 0) == ac.ERR_INVALID_ARG
    assert _status(ac.adacomp_recurrence_set_timeout_ns, h, 0) == ac.ERR_INVALID_ARG
    ac.adacomp_recurrence_set_timeout_ns(h, 10 ** 9)
    ac.adacomp_recurrence_set_fault_injection(h)


@pytest.mark.parametrize("dim", [1, 100, 2048, 4097, 8192, 8193, 2 ** 23 + 3])
@pytest.mark.parametrize("rows", [0, 1, 2, 151, 100_000])
def test_layer_norm_workspace_is_what_a_call_can_write(rows, dim):
    """Partial sums of the weight's and the bias's gradients: one per SM (152) where rows fit in
    registers, or up to 128 and a pair of sums per row; never more than there are rows."""
    h = ac.adacomp_layer_norm_init(dim, ac.BF16, ac.F32)
    sums = 8 * dim
    narrow = min(max(rows, 1), 152) * sums if dim <= 8192 else sums
    wide = min(max(rows, 1), 128) * sums + 8 * rows if dim > 4096 else sums
    assert ac.adacomp_layer_norm_backward_ws_bytes(h, rows) == max(narrow, wide)


def test_pointers_keep_the_memory_that_they_point_to():
    """A tensor whose memory is replaced afterwards (t.data = ...) is not followed, and what its
    address was taken of is not freed."""
    class OnGpu(torch.Tensor):  # passes for one; no call below reaches the GPU
        is_cuda = True

    t = torch.zeros(100).as_subclass(OnGpu)
    p = ac.adacomp_pointers([t, None])
    t.data = torch.ones(50)
    assert p.tensors[0].data_ptr() == p.array[0] != t.data_ptr()
    assert p.tensors[0].numel() == 100 and p.tensors[1] is None and not p.tensors[0].any()
