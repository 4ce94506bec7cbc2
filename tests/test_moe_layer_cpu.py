"""Host checks of the MoE layer's entry points: bad arguments are refused before any GPU work."""
import ctypes as C

from helpers import ensure_built

OK, ARG, SHAPE, DTYPE, WS = 0, 1, 2, 3, 4
P = C.c_void_p(0x1000)
ODD = C.c_void_p(0x1008)
BIG = 1 << 40


def test_sort_tokens_host_validation():
    f = ensure_built().lrm_sort_tokens
    assert f(None, P, 16, 2, 4, 64, 0, P, P, P, P, P, BIG, None, None) == ARG   # no ids
    assert f(P, None, 16, 2, 4, 64, 0, P, P, P, P, P, BIG, None, None) == ARG   # rows wanted, none given
    assert f(P, P, 16, 2, 4, 64, 0, None, P, P, P, P, BIG, None, None) == ARG
    assert f(P, P, -1, 2, 4, 64, 0, P, P, P, P, P, BIG, None, None) == ARG
    assert f(P, ODD, 16, 2, 4, 64, 0, P, P, P, P, P, BIG, None, None) == ARG
    assert f(P, P, 16, 17, 4, 64, 0, P, P, P, P, P, BIG, None, None) == SHAPE
    assert f(P, P, 16, 2, 1025, 64, 0, P, P, P, P, P, BIG, None, None) == SHAPE
    assert f(P, P, 16, 2, 4, 60, 0, P, P, P, P, P, BIG, None, None) == SHAPE
    assert f(P, P, 1 << 40, 2, 4, 64, 0, P, P, P, P, P, BIG, None, None) == SHAPE
    assert f(P, P, 16, 2, 4, 64, 2, P, P, P, P, P, BIG, None, None) == DTYPE
    assert f(P, P, 1 << 20, 2, 4, 64, 0, P, P, P, P, None, 0, None, None) == WS   # many pairs need scratch
    assert f(P, P, 1 << 20, 2, 4, 64, 0, P, P, P, P, P, 16, None, None) == WS


def test_sort_fits_the_common_workspace():
    lib = ensure_built()
    n = C.c_size_t(0)
    for T, k, E in ((1, 1, 1), (100000, 16, 1024), (50003, 6, 60)):
        assert lib.lrm_workspace_size(T, k, E, 8, 8, 0, C.byref(n)) == OK
        chunks = (T + 256 // k - 1) // (256 // k)
        common = n.value
        assert lib.lrm_sort_workspace_size(T, k, E, C.byref(n)) == OK
        assert (n.value == 0) if T * k < 10000 else (common >= n.value >= 4 * (chunks + 1) * (E + 1))
    assert lib.lrm_sort_workspace_size(1, 1, 1, None) == ARG


def test_combine_host_validation():
    lib = ensure_built()
    f = lib.lrm_combine
    assert f(None, P, P, None, 16, 2, 64, 0, 32, P, None, None) == ARG
    assert f(P, P, None, None, 16, 2, 64, 0, 32, P, None, None) == ARG
    assert f(P, P, P, ODD, 16, 2, 64, 0, 32, P, None, None) == ARG
    assert f(P, P, P, None, 16, 2, 64, 0, -1, P, None, None) == ARG
    assert f(P, P, P, None, 16, 2, 60, 0, 32, P, None, None) == SHAPE
    assert f(P, P, P, None, 16, 2, 64, 9, 32, P, None, None) == DTYPE
    assert f(None, None, None, None, 0, 2, 64, 0, 0, None, None, None) == OK   # no tokens: nothing to do
    f = lib.lrm_combine_backward
    assert f(P, P, None, P, 16, 2, 64, 0, 32, P, P, None, None) == ARG
    assert f(P, P, P, None, 16, 2, 64, 0, 32, P, P, None, None) == ARG   # dalpha needs y_s
    assert f(P, P, P, P, 16, 2, 64, 0, 32, None, P, None, None) == ARG
    assert f(P, P, P, P, 16, 0, 64, 0, 32, P, P, None, None) == ARG
    assert f(None, None, None, None, 0, 2, 64, 0, 0, None, None, None, None) == OK


def test_linear_host_validation():
    lib = ensure_built()
    n = C.c_size_t(0)
    size = lib.lrm_linear_workspace_size
    assert size(100, 4, 64, 64, 4, 0, None) == ARG
    assert size(100, 4, 64, 64, 5, 0, C.byref(n)) == ARG
    assert size(100, 4, 60, 64, 0, 0, C.byref(n)) == SHAPE
    assert size(1 << 31, 4, 64, 64, 0, 0, C.byref(n)) == SHAPE
    assert size(100, 4, 64, 64, 0, 3, C.byref(n)) == DTYPE
    assert size(100, 4, 64, 64, 4, 0, C.byref(n)) == OK and n.value > 0
    f = lib.lrm_linear
    ok = (P, P, P, P, P, 16, 4, 64, 64, 0, 0, 0, P, P, P, BIG, 0, None, None)

    def call(fn, base, **at):
        args = list(base)
        for i, v in at.items():
            args[int(i[1:])] = v
        return fn(*args)

    assert call(f, ok, a0=None) == ARG        # several experts need segments
    assert call(f, ok, a1=None) == ARG and call(f, ok, a2=None) == ARG and call(f, ok, a12=None) == ARG
    assert call(f, ok, a3=ODD) == ARG and call(f, ok, a13=ODD) == ARG
    assert call(f, ok, a5=-1) == ARG and call(f, ok, a9=7) == ARG and call(f, ok, a16=2) == ARG
    assert call(f, ok, a6=2000) == SHAPE and call(f, ok, a7=12) == SHAPE and call(f, ok, a8=4) == SHAPE
    assert call(f, ok, a10=4) == DTYPE and call(f, ok, a11=4) == DTYPE
    assert call(f, ok, a10=1, a11=0) == DTYPE  # fp32 inputs give fp32
    assert call(f, ok, a11=1) == DTYPE         # a residual with an fp32 y of bf16 inputs
    assert call(f, ok, a10=1, a11=1, a14=None) == WS and call(f, ok, a10=1, a11=1, a15=0) == WS
    assert f(None, None, P, None, None, 0, 1, 64, 64, 0, 0, 0, None, None, P, BIG, 0, None, None) == OK
    f = lib.lrm_act_backward
    ok = (P, P, P, 16, 4, 64, 1, 0, P, P, P, BIG, None, None)
    assert call(f, ok, a0=None) == ARG and call(f, ok, a1=None) == ARG and call(f, ok, a2=None) == ARG
    assert call(f, ok, a8=None) == ARG and call(f, ok, a6=-1) == ARG and call(f, ok, a9=ODD) == ARG
    assert call(f, ok, a5=4) == SHAPE and call(f, ok, a7=5) == DTYPE and call(f, ok, a11=8) == WS
    f = lib.lrm_linear_backward
    ok = (P, P, P, P, 16, 4, 64, 64, 0, P, P, P, BIG, 0, None, None)
    assert call(f, ok, a0=None) == ARG and call(f, ok, a1=None) == ARG and call(f, ok, a2=None) == ARG
    assert call(f, ok, a3=None) == ARG and call(f, ok, a9=None, a10=None) == ARG and call(f, ok, a13=9) == ARG
    assert call(f, ok, a6=63) == SHAPE and call(f, ok, a8=2) == DTYPE and call(f, ok, a11=None) == WS
