"""Host checks of the 8-bit operators and the optimiser: bad arguments are refused before any GPU work."""
import ctypes as C

from helpers import ensure_built

OK, ARG, SHAPE, DTYPE, WS = 0, 1, 2, 3, 4
P, ODD, BYTE = C.c_void_p(0x1000), C.c_void_p(0x1008), C.c_void_p(0x1002)
BIG = 1 << 40
NAN = float("nan")


def call(fn, base, **at):
    args = list(base)
    for i, v in at.items():
        args[int(i[1:])] = v
    return fn(*args)


def test_quantize():
    f = ensure_built().lrm_fp8_quantize
    ok = (P, P, 16, 2, 64, 0, 32, P, P, None, None)  # x, rows, T, k, K, dt, cap, q, scale
    for bad in (dict(a0=None), dict(a7=None), dict(a8=None), dict(a0=ODD), dict(a7=ODD), dict(a8=BYTE), dict(a1=BYTE),
                dict(a2=-1), dict(a3=0), dict(a4=0), dict(a6=-1), dict(a6=BIG)):
        assert call(f, ok, **bad) == ARG, bad
    for bad in (dict(a3=17), dict(a4=72), dict(a4=1 << 25), dict(a2=BIG)):
        assert call(f, ok, **bad) == SHAPE, bad
    assert call(f, ok, a5=2) == DTYPE
    assert call(f, ok, a1=None) == ARG          # k = 2 without rows
    assert call(f, ok, a1=None, a3=1, a6=15) == ARG  # fewer rows than tokens
    assert f(None, None, 0, 1, 64, 0, 0, None, None, None, None) == OK
    assert f(None, None, 0, 2, 64, 0, 0, None, None, None, None) == OK
    f = ensure_built().lrm_fp8_quantize_weight
    ok = (P, 4, 64, 64, 0, P, P, None)
    for bad in (dict(a0=None), dict(a5=None), dict(a6=None), dict(a0=ODD), dict(a5=ODD), dict(a6=BYTE), dict(a1=0),
                dict(a2=0), dict(a3=-16)):
        assert call(f, ok, **bad) == ARG, bad
    for bad in (dict(a1=2049), dict(a3=72), dict(a2=1 << 25), dict(a1=2048, a2=1 << 24, a3=1 << 24)):
        assert call(f, ok, **bad) == SHAPE, bad
    assert call(f, ok, a4=5) == DTYPE


def test_products():
    lib = ensure_built()
    f = lib.lrm_fp8_linear
    ok = (P, P, P, P, P, P, P, 16, 4, 64, 64, 0, P, P, None, None)
    for bad in (dict(a0=None), dict(a1=None), dict(a2=None), dict(a3=None), dict(a4=None), dict(a12=None), dict(a1=ODD),
                dict(a3=ODD), dict(a5=ODD), dict(a6=ODD), dict(a12=ODD), dict(a13=ODD), dict(a2=BYTE), dict(a4=BYTE),
                dict(a0=BYTE), dict(a7=-1), dict(a8=0), dict(a9=0), dict(a10=0), dict(a11=5), dict(a11=-1)):
        assert call(f, ok, **bad) == ARG, bad
    for bad in (dict(a7=(1 << 31) - 1), dict(a8=1025), dict(a9=12), dict(a9=1 << 25), dict(a10=72), dict(a10=1 << 25)):
        assert call(f, ok, **bad) == SHAPE, bad
    assert f(None, None, None, P, P, None, None, 0, 1, 64, 64, 4, None, None, None, None) == OK
    f = lib.lrm_fp8_linear_backward
    ok = (P, P, P, P, P, 16, 4, 64, 64, 1, P, None, None)
    for bad in (dict(a0=None), dict(a1=None), dict(a2=None), dict(a3=None), dict(a4=None), dict(a10=None), dict(a1=ODD),
                dict(a3=ODD), dict(a10=ODD), dict(a2=BYTE), dict(a4=BYTE), dict(a5=-1), dict(a9=2)):
        assert call(f, ok, **bad) == ARG, bad
    for bad in (dict(a7=72), dict(a8=72), dict(a6=1025)):
        assert call(f, ok, **bad) == SHAPE, bad
    assert f(None, None, None, P, P, 0, 1, 64, 64, 0, None, None, None) == OK


def test_adamw():
    from pruned_expert_backward_gb300 import _lib as L
    lib = ensure_built()
    size = C.c_size_t(0)

    def tensors(count=2, **over):
        t = (L.AdamwTensor * count)()
        for i in range(count):
            for name in ("w", "copy", "g", "m", "v", "m_scale", "v_scale"):
                setattr(t[i], name, 0x1000)
            t[i].n, t[i].lr_scale = 100, 1.0
        for name, v in over.items():
            setattr(t[count - 1], name, v)
        return t

    def hyper(**over):
        h = L.AdamwHyper(1e-3, 0.9, 0.95, 1e-8, 1, 0, 0.0, None, None, None)
        for name, v in over.items():
            setattr(h, name, v)
        return C.byref(h)

    def step(t, w=1, g=1, bits=8, copy=1, h=None, count=2):
        return lib.lrm_adamw(t, count, w, g, bits, copy, hyper() if h is None else h, None)

    for name in ("w", "copy", "g", "m", "v", "m_scale", "v_scale"):
        assert step(tensors(**{name: None})) == ARG, name
        assert step(tensors(**{name: 0x1002})) == ARG, name
    assert step(tensors(n=-1)) == ARG and step(tensors(n=1 << 41)) == SHAPE
    assert step(None) == ARG and step(tensors(), count=-1) == ARG
    assert step(tensors(), bits=16) == ARG and step(tensors(), copy=2) == ARG
    assert step(tensors(), w=3) == DTYPE and step(tensors(), g=3) == DTYPE
    assert step(tensors(), w=0) == DTYPE  # a copy of bf16 weights
    assert lib.lrm_adamw(tensors(), 2, 1, 1, 8, 1, None, None) == ARG
    for bad in (dict(lr=-1.0), dict(lr=NAN), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.5), dict(beta2=NAN),
                dict(eps=-1e-8), dict(grad_norm=0x1000, max_norm=0.0), dict(grad_norm=0x1000, max_norm=NAN),
                dict(grad_norm=0x1002, max_norm=1.0), dict(lr_dev=0x1002), dict(step_dev=0x1002)):
        assert step(tensors(), h=hyper(**bad)) == ARG, bad
    assert step(tensors(), h=hyper(step=0)) == SHAPE and step(tensors(), h=hyper(step=1 << 31)) == SHAPE
    # tensors without elements need no addresses, and none at all is nothing to do
    empty = (L.AdamwTensor * 2)()
    assert step(empty) == OK and step(None, count=0) == OK
    f = lib.lrm_grad_norm_workspace_size
    assert f(tensors(), 2, None) == ARG and f(None, 2, C.byref(size)) == ARG
    assert f(tensors(n=-1), 2, C.byref(size)) == ARG
    assert f(tensors(), 2, C.byref(size)) == OK and size.value >= 16
    many = tensors(1000)
    assert f(many, 1000, C.byref(size)) == OK and size.value >= 8 * 1000
    f = lib.lrm_grad_norm
    for g in (None, 0x1008):
        assert f(tensors(g=g), 2, 1, P, P, 256, None, None) == ARG
    assert f(tensors(), 2, 1, None, P, 256, None, None) == ARG and f(tensors(), 2, 1, BYTE, P, 256, None, None) == ARG
    assert f(tensors(), 2, 4, P, P, 256, None, None) == DTYPE
    assert f(tensors(), 2, 1, P, None, 256, None, None) == WS and f(tensors(), 2, 1, P, P, 8, None, None) == WS
