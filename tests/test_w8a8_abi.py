"""Refusals of the int8-activation entry points, on the host before any CUDA
call (no GPU needed)."""
import ctypes

import pytest

A, B, C, D, E, F, G, H = (ctypes.c_void_p(0x10000000 * i) for i in range(1, 9))


def at(p, off):
    return ctypes.c_void_p(p.value + off)


def test_quantize_per_token_rejects_bad_arguments(w8lib):
    f = w8lib.w8_quantize_per_token
    ok = [A, 1, 64, 4, 64, B, 64, C, D, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_1=2) == -4
    for kw in (dict(_3=-1), dict(_4=0), dict(_4=60), dict(_2=56), dict(_6=48), dict(_6=72), dict(_3=1 << 31),
               dict(_2=1 << 41), dict(_6=1 << 41)):
        assert call(**kw) == -2, kw
    for i in (0, 5, 7, 8):
        assert call(**{f"_{i}": None}) == -1
        assert call(**{f"_{i}": at(ok[i], 8)}) == -3
    assert call(_2=68) == -3                       # rows not on 16-byte boundaries
    assert call(_2=68, _3=1) != -3                 # one row has none to keep
    assert call(_5=at(A, 16)) == -8
    assert call(_7=at(A, 3 * 128)) == -8           # inside X's last row
    assert call(_8=at(B, 3 * 64 + 48)) == -8       # inside q's last row
    assert call(_8=C) == -8
    assert f(None, 1, 64, 0, 64, None, 64, None, None, None) == 0


def test_swiglu_quantize_per_token_rejects_bad_arguments(w8lib):
    f = w8lib.w8_swiglu_quantize_per_token
    assert f(A, 120, 4, 64, B, 64, C, D, None) == -2        # rows shorter than 2K
    assert f(A, 128, 4, 60, B, 64, C, D, None) == -2
    assert f(None, 128, 4, 64, B, 64, C, D, None) == -1
    assert f(A, 128, 4, 64, at(A, 3 * 256 + 128), 64, C, D, None) == -8
    assert f(A, 128, 0, 64, B, 64, C, D, None) == 0


def test_linear_rejects_bad_arguments(w8lib):
    f = w8lib.w8a8_linear
    ok = [A, 128, B, C, D, E, None, None, F, 4, 128, 256, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    for kw in (dict(_9=-1), dict(_10=0), dict(_10=124), dict(_11=0), dict(_11=252), dict(_10=65544, _1=65552),
               dict(_1=112), dict(_1=136), dict(_9=1 << 31)):
        assert call(**kw) == -2, kw
    for i in (0, 2, 3, 4, 5, 8):
        assert call(**{f"_{i}": None}) == -1
        assert call(**{f"_{i}": at(ok[i], 4)}) == -3
    assert call(_6=at(G, 1)) == -3 and call(_7=at(G, 2)) == -3
    assert call(_8=at(A, 256)) == -8 and call(_8=at(D, 16)) == -8 and call(_8=E) == -8
    assert call(_6=F) == -8 and call(_7=F) == -8
    assert call(_9=0) == 0
    assert f(None, 128, None, None, D, E, None, None, None, 0, 128, 256, None) == 0


def test_grouped_rejects_bad_arguments(w8lib):
    f = w8lib.w8a8_linear_grouped
    ok = [A, 128, B, C, G, 2, D, E, None, None, F, 4, 128, 256, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    for kw in (dict(_5=0), dict(_5=1025), dict(_11=(1 << 24) + 1), dict(_12=65544, _1=65552), dict(_13=4)):
        assert call(**kw) == -2, kw
    assert call(_4=None) == -1
    assert call(_4=at(G, 4)) == -3
    assert call(_10=at(D, 2 * 2 * 2 * 8192 - 16)) == -8     # inside the second weight
    assert call(_10=at(G, -16)) == -8
    assert call(_11=0) == 0


def test_well_formed_calls_need_a_device(w8lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert w8lib.w8_quantize_per_token(A, 1, 64, 4, 64, B, 64, C, D, None) == -6
    assert w8lib.w8a8_linear(A, 128, B, C, D, E, None, None, F, 4, 128, 256, None) == -6
    assert w8lib.w8a8_linear_grouped(A, 128, B, C, G, 2, D, E, None, None, F, 4, 128, 256, None) == -6
