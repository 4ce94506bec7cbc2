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


FORWARD, ACT_BACKWARD, DX, DW = 1, 2, 4, 8


def size_for(uses, R, E, N, K, act=NONE, dt=BF16):
    n = C.c_size_t(0)
    st = ensure_built().lrm_linear_workspace_size_for(uses, R, E, N, K, act, dt, C.byref(n))
    assert st == OK
    return n.value


def test_scratch_is_what_the_call_uses():
    """One call's scratch counts neither the other calls' nor planes that the one-pass kernel does not form."""
    mb = 1 << 20
    # a generated token's and 64 tokens' experts' products in fp32: weights of 1.6 GB and more are not split
    for R, N, K in ((8, 768, 2048), (8, 1408, 4096), (512, 768, 2048)):
        assert 0 < size_for(FORWARD, R, 128, N, K, SWIGLU, F32) <= 4096
    assert 0 < size_for(FORWARD, 8, 1, 4096, 4096, NONE, F32) <= 4096
    # more rows: x and w as three bf16 planes
    for R, E, N, K in ((4096, 4, 256, 512), (32, 1, 256, 512)):
        assert size_for(FORWARD, R, E, N, K, NONE, F32) >= 6 * (R * K + E * N * K)
    # bias sums: a partial sum per 128 rows and expert, whatever the type
    for dt in (BF16, F32):
        assert 4 * (512 + 1) * 2048 <= size_for(ACT_BACKWARD, 65536, 1, 2048, 2048, NONE, dt) <= 8 * mb
    # either gradient alone: dz and one other operand in planes
    R, N, K = 4096, 512, 1024
    dx, dw = (size_for(u, R, 1, N, K, NONE, F32) for u in (DX, DW))
    assert 6 * (R * N + N * K) <= dx <= 6 * (R * N + N * K) + 8 * mb
    assert 6 * (R * N + R * K) <= dw <= 6 * (R * N + R * K) + 32 * mb  # and sums of parts of the rows
    assert max(dx, dw) < size_for(DX | DW, R, 1, N, K, NONE, F32) <= dx + dw
    # a buffer for all of them is the one that lrm_linear_workspace_size gives
    for act in (NONE, SWIGLU):
        for dt in (BF16, F32):
            for R, E, N, K in ((0, 4, 64, 72), (8, 128, 768, 2048), (3000, 3, 136, 264), (9000, 2, 72, 328)):
                every = [size_for(u, R, E, N, K, act, dt) for u in (FORWARD, ACT_BACKWARD, DX | DW)]
                assert size(R, E, N, K, act, dt) == max(every) == size_for(15, R, E, N, K, act, dt)


def test_scratch_size_refusals():
    f, n = ensure_built().lrm_linear_workspace_size_for, C.c_size_t(0)
    assert f(0, 100, 4, 64, 64, 0, 0, C.byref(n)) == ARG and f(16, 100, 4, 64, 64, 0, 0, C.byref(n)) == ARG
    assert f(1, 100, 4, 64, 64, 0, 0, None) == ARG and f(1, 100, 4, 64, 64, 5, 0, C.byref(n)) == ARG
    assert f(1, 100, 4, 60, 64, 0, 0, C.byref(n)) == SHAPE and f(1, 100, 4, 64, 64, 0, 2, C.byref(n)) == DTYPE


def test_most_rows():
    """Row numbers of a tile past the last row stay in 32 bits: 1023 rows below INT32_MAX are the most."""
    lib, n = ensure_built(), C.c_size_t(0)
    most = (1 << 31) - 1024
    for E in (1, 4):
        assert size(most, E, 8, 8) > 0
        for R in (most + 1, (1 << 31) - 1):
            assert lib.lrm_linear_workspace_size(R, E, 8, 8, NONE, BF16, C.byref(n)) == SHAPE
            assert lib.lrm_linear(P, P, P, None, None, R, E, 8, 8, NONE, 0, 0, P, None, P, BIG, 0, None, None) == SHAPE
            assert lib.lrm_linear_backward(P, P, P, P, R, E, 8, 8, 0, P, P, P, BIG, 0, None, None) == SHAPE
            assert lib.lrm_act_backward(P, P, P, R, E, 8, NONE, 0, P, P, P, BIG, None, None) == SHAPE


def test_kernels_check_their_own_indices():
    """Every source file of the layer's kernels that writes by an index of its own has checks for the debug build."""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc = os.path.join(root, "pruned_expert_backward_gb300", "csrc")
    for name in ("permute.cu", "act_backward.cu", "linear_rows.cu", "linear_simt.cu", "linear_tc.cu"):
        assert "LRM_DCHECK(" in open(os.path.join(csrc, name)).read(), name


def test_scratch_size_of_a_type_that_is_not_supported():
    """The binding refuses other types; it answered for fp32."""
    import torch

    import pruned_expert_backward_gb300 as lrm
    assert lrm.lrm_linear_workspace_size(100, 4, 64, 64, "swiglu", torch.bfloat16) > 0
    for dtype in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(TypeError):
            lrm.lrm_linear_workspace_size(100, 4, 64, 64, "swiglu", dtype)
