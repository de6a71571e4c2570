"""Host-side checks of the linear layers' and vocabulary losses' entry points (no GPU): argument errors come back
before any launch."""
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


def _caller(call, good):
    def with_(**change):
        args = list(good)
        for k, v in change.items():
            args[int(k[1:])] = v
        return call(*args)
    return with_


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "adacomp.h")).read()
    assert int(re.search(r"#define ADACOMP_MAX_TEACHER (\d+)", text).group(1)) == ac.MAX_TEACHER
    for name in ("NONE", "RELU", "GELU", "GELU_TANH", "SILU"):
        assert int(re.search(rf"ADACOMP_ACT_{name} = (\d+)", text).group(1)) == getattr(ac, f"ACT_{name}")


@pytest.mark.parametrize("args", [(0, 4, 0, 0), (4, 0, 0, 0), (-1, 4, 0, 0), (2 ** 31, 4, 0, 0), (4, 2 ** 31, 0, 0),
                                  (4, 4, 2, 0), (4, 4, 0, -1), (4, 4, 0, 5)])
def test_linear_init_refuses(args):
    p = ctypes.c_void_p(5)
    assert ac.lib().adacomp_linear_init(ctypes.byref(p), *args) == ac.ERR_INVALID_ARG
    assert p.value is None
    assert ac.lib().adacomp_linear_init(None, 4, 4, 0, 0) == ac.ERR_INVALID_ARG


@pytest.mark.parametrize("args", [(0, 4, 0), (4, 0, 0), (4, -1, 0), (2 ** 31, 4, 0), (4, 2 ** 31, 0), (4, 4, 2)])
def test_vocab_init_refuses(args):
    p = ctypes.c_void_p(5)
    assert ac.lib().adacomp_vocab_init(ctypes.byref(p), *args) == ac.ERR_INVALID_ARG
    assert p.value is None


def test_sizes_of_nothing():
    h, v = ac.adacomp_linear_init(8, 8), ac.adacomp_vocab_init(8, 8)
    for rows in (-1, 2 ** 31):
        assert ac.adacomp_linear_forward_ws_bytes(h, rows) == ac.adacomp_linear_backward_ws_bytes(h, rows) == 0
        assert ac.adacomp_vocab_loss_forward_ws_bytes(v, rows) == ac.adacomp_vocab_loss_backward_ws_bytes(v, rows) == 0
    for k in (0, ac.MAX_TEACHER + 1):
        assert ac.adacomp_distill_forward_ws_bytes(v, 5, k) == ac.adacomp_distill_backward_ws_bytes(v, 5, k) == 0
    assert ac.adacomp_vocab_loss_backward_ws_bytes(v, 5) <= ac.adacomp_distill_backward_ws_bytes(v, 5, 100)


@pytest.mark.parametrize("dt", [ac.F32, ac.BF16])
def test_linear_forward_refuses_before_launch(dt):
    h = ac.adacomp_linear_init(10, 6, dt, ac.ACT_GELU)
    need = ac.adacomp_linear_forward_ws_bytes(h, 4)
    call = _caller(ac.lib().adacomp_linear_forward, [h.ptr, 4, A, 10, A, 10, A, A, 6, A, 6, A, 6, A, need, None])
    for change in ({"a0": None}, {"a1": -1}, {"a1": 2 ** 31}, {"a2": None}, {"a3": -1}, {"a4": None}, {"a5": -1},
                   {"a8": -1}, {"a9": None}, {"a10": 5}, {"a12": 5}, {"a13": None}):
        assert call(**change) == ac.ERR_INVALID_ARG, change
    for place in (2, 4, 6, 7, 9, 11):
        assert call(**{f"a{place}": A + 1}) == ac.ERR_ALIGNMENT, place
    assert call(a13=A + 8) == ac.ERR_ALIGNMENT
    if need:
        assert call(a14=need - 1) == ac.ERR_WORKSPACE
    assert call(a1=0, a2=None, a9=None) == ac.OK


@pytest.mark.parametrize("dt", [ac.F32, ac.BF16])
def test_linear_backward_refuses_before_launch(dt):
    h = ac.adacomp_linear_init(10, 6, dt, ac.ACT_GELU)
    need = ac.adacomp_linear_backward_ws_bytes(h, 4)
    call = _caller(ac.lib().adacomp_linear_backward,
                   [h.ptr, 4, A, 6, A, 10, A, 10, A, 6, A, 10, A, 10, A, A, need, None])
    for change in ({"a0": None}, {"a1": -1}, {"a1": 2 ** 31}, {"a2": None}, {"a3": -1}, {"a4": None}, {"a5": -1},
                   {"a6": None}, {"a7": -1}, {"a8": None}, {"a9": -1}, {"a11": 9}, {"a13": 9}, {"a15": None},
                   {"a10": None, "a12": None, "a14": None}):
        assert call(**change) == ac.ERR_INVALID_ARG, change
    for place in (2, 4, 6, 8, 10, 12, 14):
        assert call(**{f"a{place}": A + 1}) == ac.ERR_ALIGNMENT, place
    assert call(a15=A + 8) == ac.ERR_ALIGNMENT
    assert call(a16=need - 1) == ac.ERR_WORKSPACE


@pytest.mark.parametrize("dt", [ac.F32, ac.BF16])
def test_vocab_loss_refuses_before_launch(dt):
    h, L = ac.adacomp_vocab_init(10, 60, dt), ac.lib()
    need = ac.adacomp_vocab_loss_forward_ws_bytes(h, 4)
    call = _caller(L.adacomp_vocab_loss_forward, [h.ptr, 4, A, 10, A, 10, A, 8, A, A, A, need, None])
    for change in ({"a0": None}, {"a1": -1}, {"a1": 2 ** 31}, {"a2": None}, {"a3": -1}, {"a4": None}, {"a5": -1},
                   {"a6": None}, {"a7": 2}, {"a8": None}, {"a9": None}, {"a10": None}):
        assert call(**change) == ac.ERR_INVALID_ARG, change
    for change in ({"a2": A + 1}, {"a4": A + 1}, {"a6": A + 4}, {"a8": A + 2}, {"a9": A + 2}, {"a10": A + 8}):
        assert call(**change) == ac.ERR_ALIGNMENT, change
    assert call(a11=need - 1) == ac.ERR_WORKSPACE
    assert call(a1=0, a2=None, a6=None) == ac.OK
    need = ac.adacomp_vocab_loss_backward_ws_bytes(h, 4)
    call = _caller(L.adacomp_vocab_loss_backward,
                   [h.ptr, 4, A, 10, A, 10, A, 4, A, A, 1, A, 10, A, 10, A, need, None])
    for change in ({"a0": None}, {"a1": -1}, {"a2": None}, {"a4": None}, {"a6": None}, {"a7": 1}, {"a8": None},
                   {"a9": None}, {"a10": -1}, {"a12": 9}, {"a14": 9}, {"a11": None, "a13": None}, {"a15": None}):
        assert call(**change) == ac.ERR_INVALID_ARG, change
    for change in ({"a2": A + 1}, {"a4": A + 1}, {"a6": A + 2}, {"a8": A + 2}, {"a9": A + 2}, {"a11": A + 1},
                   {"a13": A + 1}, {"a15": A + 8}):
        assert call(**change) == ac.ERR_ALIGNMENT, change
    assert call(a16=need - 1) == ac.ERR_WORKSPACE


@pytest.mark.parametrize("dt", [ac.F32, ac.BF16])
def test_distill_refuses_before_launch(dt):
    h, L = ac.adacomp_vocab_init(10, 60, dt), ac.lib()
    need = ac.adacomp_distill_forward_ws_bytes(h, 4, 5)
    call = _caller(L.adacomp_distill_forward, [h.ptr, 4, A, 10, A, 10, 5, A, 5, A, 5, dt, 2.0, A, A, A, need, None])
    backward_need = ac.adacomp_distill_backward_ws_bytes(h, 4, 5)
    backward = _caller(L.adacomp_distill_backward,
                       [h.ptr, 4, A, 10, A, 10, 5, A, 5, A, 5, dt, 2.0, A, A, 1, A, 10, A, 10, A, backward_need, None])
    inf, nan = float("inf"), float("nan")
    for change in ({"a0": None}, {"a1": -1}, {"a2": None}, {"a4": None}, {"a6": 0}, {"a6": 257}, {"a7": None},
                   {"a8": -1}, {"a9": None}, {"a10": -1}, {"a11": 2}, {"a12": 0.0}, {"a12": -1.0}, {"a12": inf}, {"a12": 1e-39}, {"a12": 1e20},
                   {"a12": nan}, {"a13": None}, {"a14": None}):
        assert call(**change) == ac.ERR_INVALID_ARG, change
        assert backward(**change) == ac.ERR_INVALID_ARG, change
    assert backward(a16=None, a18=None) == backward(a15=-1) == backward(a17=9) == backward(a19=9) == ac.ERR_INVALID_ARG
    for change in ({"a2": A + 1}, {"a4": A + 1}, {"a7": A + 2}, {"a9": A + 1}, {"a13": A + 2}):
        assert call(**change) == backward(**change) == ac.ERR_ALIGNMENT, change
    assert backward(a16=A + 1) == backward(a18=A + 1) == backward(a20=A + 8) == ac.ERR_ALIGNMENT
    assert call(a16=need - 1) == backward(a21=backward_need - 1) == ac.ERR_WORKSPACE


def test_the_binding_refuses_tensors_that_do_not_fit():
    h, v = ac.adacomp_linear_init(10, 6), ac.adacomp_vocab_init(10, 60)
    x, w, y = torch.zeros(4, 10), torch.zeros(6, 10), torch.zeros(4, 6)
    for args in ((x, w, y, y), (x[:, :9], w, y, y), (x.bfloat16(), w, y, y)):
        with pytest.raises(ValueError):
            ac.adacomp_linear_forward(h, *args)
    with pytest.raises(ValueError):
        ac.adacomp_linear_backward(h, y, x, w, y, dx=x)
    one = torch.zeros(4)
    for target in (one, one.long(), one.to(torch.int16)):
        with pytest.raises(ValueError):
            ac.adacomp_vocab_loss_forward(v, x, torch.zeros(60, 10), target, one, one, one)
    with pytest.raises(ValueError):
        ac.adacomp_distill_forward(v, x, torch.zeros(60, 10), one.int(), one, 1.0, one, one, one)


def test_free_takes_null_and_twice():
    for name in ("linear", "vocab"):
        getattr(ac.lib(), f"adacomp_{name}_free")(None)
    h, v = ac.adacomp_linear_init(10, 6), ac.adacomp_vocab_init(10, 60)
    for _ in range(2):
        ac.adacomp_linear_free(h)
        ac.adacomp_vocab_free(v)


@pytest.mark.parametrize("dim,vocab", [(1, 1), (8, 1000), (64, 2047), (2048, 50304), (500, 10007)])
@pytest.mark.parametrize("dt", [ac.F32, ac.BF16])
def test_a_workspace_for_more_rows_is_enough_for_fewer(dim, vocab, dt):
    """Fewer rows take the vocabulary in larger pieces, and split sums into more parts."""
    v, h = ac.adacomp_vocab_init(dim, vocab, dt), ac.adacomp_linear_init(dim, vocab, dt)
    rows = sorted({1, 2, 127, 128, 129, 1000, 2500, 4096, 5000, 5120, 8191, 8192, 65536, 65537, 131072, 134016, 134144, 10 ** 6})
    for size in (lambda r: ac.adacomp_vocab_loss_forward_ws_bytes(v, r), lambda r: ac.adacomp_vocab_loss_backward_ws_bytes(v, r),
                 lambda r: ac.adacomp_distill_forward_ws_bytes(v, r, 9), lambda r: ac.adacomp_distill_backward_ws_bytes(v, r, 9),
                 lambda r: ac.adacomp_linear_forward_ws_bytes(h, r), lambda r: ac.adacomp_linear_backward_ws_bytes(h, r)):
        sizes = [size(r) for r in rows]
        assert sizes == sorted(sizes) and sizes[0] > 0
