"""Host checks of the MoE layer's entry points at their limits: no rows, the largest sizes, scratch sizes."""
import ctypes as C

import pytest

from helpers import ensure_built

OK, ARG, SHAPE, DTYPE, WS = 0, 1, 2, 3, 4
P = C.c_void_p(0x1000)
BIG = 1 << 40
BF16, F32 = 0, 1
NONE, SWIGLU = 0, 4


def size(R, E, N, K, act=NONE, dt=BF16):
    n = C.c_size_t(0)
    st = ensure_built().lrm_linear_workspace_size(R, E, N, K, act, dt, C.byref(n))
    assert st == OK
    return n.value


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("E", [1, 4, 1024])
def test_no_rows(E, dt):
    """An expert shard without a token: the sizes and the calls answer, nothing is launched."""
    lib = ensure_built()
    assert size(0, E, 64, 72, NONE, dt) > 0 and size(0, E, 64, 72, SWIGLU, dt) > 0
    seg = P if E > 1 else None
    assert lib.lrm_linear(seg, None, P, None, None, 0, E, 64, 72, NONE, dt, dt, None, None, P, BIG, 0, None, None) == OK
    assert lib.lrm_linear_backward(seg, None, None, P, 0, E, 64, 72, dt, P, None, P, BIG, 0, None, None) == OK
    assert lib.lrm_act_backward(seg, None, None, 0, E, 64, SWIGLU, dt, None, None, None, 0, None, None) == OK
