"""GPU checks of the MoE layer's entry points at their limits, against 64-bit plain forms.

Tolerances as in test_moe_layer_gpu.py, whose checks are used here."""
import pytest
import torch

from helpers import ensure_built
from test_moe_layer_gpu import BF16, EPS, F32, act64, check, check_linear, gen, linear_inputs, randn, routing, segments

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


@pytest.fixture
def status():
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    yield st
    torch.cuda.synchronize()
    assert int(st.item()) == 0


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("E", [None, 1, 5])
def test_no_rows(E, dt, status):
    """A product without rows: empty outputs, weight and bias gradients of zeros."""
    import pruned_expert_backward_gb300 as lrm
    lead, seg = ((), None) if E is None else ((E,), torch.zeros(E + 1, dtype=torch.int32, device="cuda"))
    x, w, b = randn(gen(0), 0, 72, dt=dt), randn(gen(1), *lead, 64, 72, dt=dt), randn(gen(2), *lead, 64, dt=dt)
    y, z = lrm.lrm_linear(x, w, bias=b, act="swiglu", seg_offsets=seg, save_z=True, dev_status=status)
    assert y.shape == (0, 32) and z.shape == (0, 64)
    dw, db = torch.full((*lead, 64, 72), 7.0, device="cuda"), torch.full((*lead, 64), 7.0, device="cuda")
    dz, _ = lrm.lrm_act_backward(y, z, act="swiglu", seg_offsets=seg, db=db, dev_status=status)
    dx, _ = lrm.lrm_linear_backward(dz, x, w, seg_offsets=seg, dw=dw, dev_status=status)
    assert dz.shape == (0, 64) and dx.shape == (0, 72)
    assert torch.count_nonzero(db) == 0 and torch.count_nonzero(dw) == 0


def test_layer_without_tokens():
    import pruned_expert_backward_gb300 as lrm
    for dt in (BF16, F32):
        layer = lrm.MoeLayer(0, 2, 4, 64, 32, dtype=dt)
        idx, alpha = torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, 2, device="cuda")
        x, wg, wd = randn(gen(0), 0, 64, dt=dt), randn(gen(1), 4, 64, 64, dt=dt), randn(gen(2), 4, 64, 32, dt=dt)
        assert layer.forward(x, idx, alpha, wg, wd).shape == (0, 64)
        dx, dalpha, dwg, dwd = layer.backward(x, alpha, wg, wd)
        assert dx.shape == (0, 64) and dalpha.shape == (0, 2)
        assert torch.count_nonzero(dwg) == 0 and torch.count_nonzero(dwd) == 0
        assert int(layer.dev_status.item()) == 0


def test_few_fp32_rows_take_no_planes(status):
    """fp32 products of few rows, and any on the CUDA cores, run with 256 bytes of scratch, dense and per expert."""
    import pruned_expert_backward_gb300 as lrm
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for R, E, simt in ((8, None, 0), (24, None, 0), (8, 16, 0), (100, 16, 0), (200, None, 1), (200, 3, 1)):
        g = gen(R)
        seg = segments("ragged", R, E, g) if E else None
        x, w, b, res = linear_inputs(g, F32, R, 80, 40, 136, True, True, E)
        y, z = lrm.lrm_linear(x, w, bias=b, residual=res, act="swiglu", seg_offsets=seg, save_z=True, ws=small,
                              flags=simt, dev_status=status)
        check_linear(x, w, b, res, "swiglu", seg, y, z)
    x, w = randn(gen(1), 200, 136, dt=F32), randn(gen(2), 80, 136, dt=F32)
    with pytest.raises(lrm.LrmError):  # the tiles need the planes
        lrm.lrm_linear(x, w, ws=small)


def test_calls_allocate_what_they_use():
    """Scratch made by the binding: none that belongs to another call of the layer."""
    import pruned_expert_backward_gb300 as lrm

    def peak(call):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        out = call()
        torch.cuda.synchronize()
        made = sum(t.numel() * t.element_size() for t in out if t is not None)
        return torch.cuda.max_memory_allocated() - before - made

    mb = 1 << 20
    dy, z = torch.zeros(16384, 512, device="cuda"), torch.zeros(16384, 512, device="cuda")
    assert peak(lambda: lrm.lrm_act_backward(dy, z, act="silu")) <= 2 * mb
    seg = torch.zeros(65, dtype=torch.int32, device="cuda")
    x, w = torch.zeros(8, 512, device="cuda"), torch.zeros(64, 256, 512, device="cuda")
    assert peak(lambda: lrm.lrm_linear(x, w, seg_offsets=seg)) <= 2 * mb
    x, w = torch.zeros(4096, 512, device="cuda"), torch.zeros(512, 512, device="cuda")
    assert peak(lambda: lrm.lrm_linear_backward(x, x, w, need_dw=False)) <= 6 * (4096 + 512) * 512 + 8 * mb
    served = lrm.MoeLayer(1, 8, 128, 2048, 768, dtype=F32, train=False)
    assert served.ws.numel() <= mb


def test_sort_of_no_tokens_with_rows_given(status):
    """T = 0 through the C ABI with buffers at hand: the segments come out empty, in every form and width."""
    lib = ensure_built()
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = buf.data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    for E in (4, 300, 1024):
        for H in (8, 512, 4096):
            for dt in (0, 1):
                seg = torch.full((E + 1,), 7, dtype=torch.int32, device="cuda")
                st = lib.lrm_sort_tokens(p, p, 0, 2, E, H, dt, seg.data_ptr(), p, p, p, p, buf.numel(),
                                         status.data_ptr(), stream)
                assert st == 0 and torch.count_nonzero(seg) == 0


@pytest.mark.parametrize("dt,N", [(F32, 8388616), (BF16, 16777216)], ids=["f32", "bf16"])
def test_act_backward_of_many_columns(dt, N, status):
    """Up to 2^24 columns: more blocks of columns than a launch grid's second dimension holds."""
    import pruned_expert_backward_gb300 as lrm
    dy, z = randn(gen(1), 2, N, dt=dt), randn(gen(2), 2, N, dt=dt)
    dz, db = lrm.lrm_act_backward(dy, z, act="relu", dev_status=status)
    want = torch.where(z > 0, dy, torch.zeros_like(dy))
    assert torch.equal(dz, want) and torch.equal(db, want[0].float() + want[1].float())


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_products_of_many_columns_on_the_cuda_cores(dt, status):
    import pruned_expert_backward_gb300 as lrm
    N = 4194320
    x, w = randn(gen(1), 3, 8, dt=dt), randn(gen(2), N, 8, dt=dt)
    y, _ = lrm.lrm_linear(x, w, flags=1, dev_status=status)
    check_linear(x, w, None, None, "none", None, y, None)
    y, _ = lrm.lrm_linear(x, w, act="swiglu", flags=1, dev_status=status)
    check_linear(x, w, None, None, "swiglu", None, y, None)
    dz = randn(gen(3), 3, N, dt=dt)
    _, dw = lrm.lrm_linear_backward(dz, x, w, need_dx=False, flags=1, dev_status=status)
    check(dw, dz.double().t() @ x.double(), 4 * EPS * (dz.double().abs().t() @ x.double().abs()))
    wt, d8 = w.t().contiguous(), randn(gen(4), 3, 8, dt=dt)
    dx, _ = lrm.lrm_linear_backward(d8, dz, wt, need_dw=False, flags=1, dev_status=status)
    check(dx, d8.double() @ wt.double(), 9 * EPS * (d8.double().abs() @ wt.double().abs()))


@pytest.mark.parametrize("dt,H", [(BF16, 33554432), (F32, 16777216)], ids=["bf16", "f32"])
def test_combine_of_wide_rows(dt, H, status):
    import pruned_expert_backward_gb300 as lrm
    row, alpha = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda"), torch.tensor([[0.5], [2.0]], device="cuda")
    y_s = randn(gen(1), 2, H, dt=dt)
    y = lrm.lrm_combine(row, alpha, y_s, dev_status=status)  # (exact: powers of two)
    assert torch.equal(y[0], y_s[1] * 0.5) and torch.equal(y[1], y_s[0] * 2)


def one_sign(g, rows, K):
    """Values of one sign, the rows scaled apart over a factor of two, so that sums round to bf16 evenly."""
    scale = 2.0 ** (torch.arange(rows, device="cuda", dtype=F32)[:, None] / rows)
    return ((torch.rand(rows, K, generator=g, device="cuda") + 0.5) * scale).to(BF16)


def bias_of(got, want):
    return ((got.double() - want) / want).mean().abs().item()


@pytest.mark.parametrize("E", [None, 3], ids=["dense", "experts"])
@pytest.mark.parametrize("R", [3, 13, 27])
def test_fp32_sums_of_few_rows(R, E, status):
    """fp32 outputs of bf16 inputs, long sums of one sign: at most 256 products in a row are added with truncation
    (16 steps of at most 2^-23 each), the rest to nearest."""
    import pruned_expert_backward_gb300 as lrm
    K, N = 65536, 64
    g = gen(R)
    x, w = one_sign(g, R, K), one_sign(g, N * (E or 1), K).view(*((E,) if E else ()), N, K)
    seg = torch.tensor([0, 0, R, R], dtype=torch.int32, device="cuda") if E else None
    y, _ = lrm.lrm_linear(x, w, seg_offsets=seg, out_dtype=F32, dev_status=status)
    want = x.double() @ (w[1] if E else w).double().t()
    assert bias_of(y, want) <= 16 * EPS


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_long_bf16_sums(act, status):
    """bf16 outputs of sums of 262144 products of one sign: the mean error is that of 5120 (SwiGLU: 2560) roundings to
    2^-9, 6 deviations of 2^-9 / sqrt 3 allowed; a truncating accumulator is 1.4e-3 off."""
    import pruned_expert_backward_gb300 as lrm
    R, N, K = 40, 128, 262144
    g = gen(7)
    x, w = one_sign(g, R, K) * 0.125, one_sign(g, N, K) * 0.125
    none = torch.empty(0, dtype=torch.uint8, device="cuda")  # (with scratch the sum would be cut into parts)
    y, _ = lrm.lrm_linear(x, w, act=act, ws=none, dev_status=status)
    want = x.double() @ w.double().t()
    if act == "swiglu":
        want = act64(want, act)
    assert bias_of(y, want) <= 6 * 2.0 ** -9 / 3 ** 0.5 / want.numel() ** 0.5 + 32 * EPS


def test_long_bf16_sums_of_the_gradient(status):
    import pruned_expert_backward_gb300 as lrm
    R, N, K = 40, 262144, 9984  # (wide enough not to be cut into parts)
    g = gen(8)
    dz, w = one_sign(g, R, N), torch.empty(N, K, dtype=BF16, device="cuda")
    want = torch.zeros(R, K, dtype=torch.float64, device="cuda")
    for i in range(0, N, 16384):
        w[i:i + 16384] = one_sign(g, K, 16384).t()
        want += dz[:, i:i + 16384].double() @ w[i:i + 16384].double()
    dx, _ = lrm.lrm_linear_backward(dz, dz[:, :K].contiguous(), w, need_dw=False, dev_status=status)
    assert bias_of(dx, want) <= 6 * 2.0 ** -9 / 3 ** 0.5 / want.numel() ** 0.5 + 32 * EPS


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_the_layer_allocates_nothing_after_the_first_call(dt):
    """MoeLayer's calls make no tensor and the library takes no device memory, trained or served; tokens enough for
    the sort to need its scratch.  Both give the same y."""
    import pruned_expert_backward_gb300 as lrm
    T, k, E, H, I = 2000, 8, 12, 136, 72
    g = gen(5)
    idx, alpha = routing(g, T, k, E, 1.0, 0.1)
    x, dy = randn(g, T, H, dt=dt), randn(g, T, H, dt=dt)
    wg, wd = randn(g, E, 2 * I, H, dt=dt, std=H ** -0.5), randn(g, E, H, I, dt=dt, std=I ** -0.5)
    layer, served = lrm.MoeLayer(T, k, E, H, I, dtype=dt), lrm.MoeLayer(T, k, E, H, I, dtype=dt, train=False)

    def step():
        y = layer.forward(x, idx, alpha, wg, wd, residual=x)
        layer.backward(dy, alpha, wg, wd)
        return y, served.forward(x, idx, alpha, wg, wd, residual=x)

    step()
    torch.cuda.synchronize()
    made, free = torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]
    y, y_served = step()
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == made
    assert torch.cuda.mem_get_info()[0] >= free
    assert torch.equal(y, y_served)
    assert int(layer.dev_status.item()) == 0 and int(served.dev_status.item()) == 0
