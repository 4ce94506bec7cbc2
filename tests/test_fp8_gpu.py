"""GPU parity of the 8-bit operators: quantisers, block-scaled product and its rows' gradient, against 64-bit forms.

Tolerances, from the arithmetic:
  * quantisers: every step is one fp32 operation rounded to nearest, so values and scales equal numpy's bit for bit.
  * products: the operands' values are taken as exact in 64 bits; the products of e4m3 values are exact in fp32, and
    the K sums and two scalings err by at most (K + 1) 2^-23 sum |a b| in any order, rounded or truncated: the
    checks of test_moe_layer_gpu.py, with bf16's half step 2^-9 doubled to 2^-8.
  * a bf16 value in 8 bits is within 2^-4 of its magnitude, or 2^-10 steps of its block's scale (subnormals).
"""
import numpy as np
import pytest
import torch

from helpers import ensure_built
from test_moe_layer_gpu import BF16, EPS, F32, check, check_linear, gen, randn, rows_of, routing, segments

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
LEAST = np.float32(2.0 ** -100)


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


def blocks(n):
    return -(-n // 128)


def plain_blocks(x, rows):
    """e4m3 values and scales of blocks of rows x 128, each step in numpy's fp32."""
    x = x.float().cpu().numpy()
    R, K = x.shape
    q, scale = np.zeros((R, K), np.float32), np.zeros((-(-R // rows), blocks(K)), np.float32)
    with np.errstate(all="ignore"):
        for i in range(scale.shape[0]):
            for j in range(scale.shape[1]):
                at = np.s_[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128]
                m = np.abs(x[at]).max()
                top = m if np.isnan(m) else np.maximum(m, LEAST)
                scale[i, j] = top / np.float32(448)
                q[at] = x[at] * (np.float32(448) / top)
    return torch.from_numpy(q).to(FP8), torch.from_numpy(scale)


def same_bits(got, want):
    """Equal values, NaN in the same places."""
    g, w = got.float().cpu(), want.float().cpu()
    assert g.shape == w.shape and torch.equal(torch.isnan(g), torch.isnan(w))
    assert torch.equal(torch.nan_to_num(g, nan=0.0), torch.nan_to_num(w, nan=0.0))


def operand(q, scale, rows, halves=1):
    """What 8-bit values [..., n, k] stand for, in 64 bits; halves: matrices below one another (rows > 1)."""
    a = q.double()
    s = scale.double().repeat_interleave(128, -1)[..., : a.shape[-1]]
    if rows == 1:
        return a * s
    s = s.unflatten(-2, (halves, -1)).repeat_interleave(128, -2)[..., : a.shape[-2] // halves, :].flatten(-3, -2)
    return a * s


def columns(q, scale, halves):
    """The same for rows whose columns come in halves."""
    R = q.shape[0]
    return operand(q.view(R * halves, -1), scale.view(R * halves, -1), 1).view(R, -1)


# ------------------------------------------------------------------------------ quantisers ------
ROWS = [(1, 16), (1, 128), (3, 144), (17, 4096), (64, 2048), (257, 112), (1000, 1040), (33, 8208)]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", ROWS, ids=str)
def test_quantize_rows(shape, dt, status):
    import pruned_expert_backward_gb300 as lrm
    g = gen(sum(shape))
    x = randn(g, *shape, dt=dt, std=3.0)
    x[0] = 0
    x[-1, : shape[1] // 2] *= 1e-30
    q, scale = lrm.lrm_fp8_quantize(x, dev_status=status)
    wq, ws = plain_blocks(x, 1)
    same_bits(scale, ws)
    same_bits(q, wq)
    value = operand(q, scale, 1)
    step = scale.double().repeat_interleave(128, 1)[:, : shape[1]] * 2.0 ** -10
    assert bool(((value - x.double()).abs() <= 2.0 ** -4 * x.double().abs() + step).all())


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_quantize_extremes(dt, status):
    """The types' lowest and smallest values, zeros, infinities and NaN: a block with one that is not finite is NaN,
    its neighbours are not."""
    import pruned_expert_backward_gb300 as lrm
    low, tiny = torch.finfo(dt).min, torch.finfo(dt).tiny
    x = torch.zeros(8, 272, dtype=dt, device="cuda")
    x[0, 3], x[0, 200] = low, 1.0
    x[1, 5], x[1, 6], x[1, 130] = tiny, -tiny, tiny / 128
    x[2, 0], x[2, 1], x[2, 140] = float("inf"), 1.0, 2.0
    x[3, 127], x[3, 128] = float("nan"), 3.0
    x[4, 256], x[4, 0] = float("-inf"), 5.0
    x[5] = 1.0
    x[5, 7] = -448.0
    q, scale = lrm.lrm_fp8_quantize(x, dev_status=status)
    wq, ws = plain_blocks(x, 1)
    same_bits(scale, ws)
    same_bits(q, wq)
    assert bool(torch.isfinite(operand(q, scale, 1)[:2]).all())
    bad = torch.isnan(operand(q, scale, 1))
    assert bool(bad[2, :128].all()) and bool(bad[3, :128].all()) and bool(bad[4, 256:].all())
    assert int(bad.sum()) == 128 + 128 + 16
    assert q[0, 3].float().item() == -448.0 and q[5, 7].float().item() == -448.0


def test_quantize_to_sorted_rows(status):
    import pruned_expert_backward_gb300 as lrm
    for T, k, E, K, masked in ((1, 8, 16, 256, 0.0), (50, 3, 7, 144, 0.3), (700, 8, 128, 1040, 0.1),
                               (40, 16, 16, 16, 0.5), (9, 1, 4, 128, 0.0)):
        g = gen(T)
        idx, _ = routing(g, T, k, E, masked=masked)
        x = randn(g, T, K)
        seg, pair, row, _ = lrm.lrm_sort_tokens(idx, None, E, dev_status=status)
        q = torch.full((T * k, K), 3.0, device="cuda").to(FP8)
        scale = torch.full((T * k, blocks(K)), 5.0, device="cuda")
        lrm.lrm_fp8_quantize(x, row_of_pair=row, k=k, q=q, scale=scale, dev_status=status)
        wq, ws = lrm.lrm_fp8_quantize(x, dev_status=status)
        n = int(seg[-1])
        same_bits(q[:n], wq.view(torch.uint8)[pair[:n].long() // k].view(FP8))
        same_bits(scale[:n], ws[pair[:n].long() // k])
        assert bool((q[n:].float() == 3.0).all()) and bool((scale[n:] == 5.0).all())  # rows of no pair are left alone


def test_quantize_bad_rows_are_skipped():
    import pruned_expert_backward_gb300 as lrm
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.ones(3, 144, device="cuda")
    q, scale = torch.zeros(4, 144, device="cuda").to(FP8), torch.zeros(4, 2, device="cuda")
    row = torch.tensor([0, -1, 4, 2, -2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    lrm.lrm_fp8_quantize(x, row_of_pair=row, k=2, q=q, scale=scale, dev_status=st)
    assert int(st.item()) == 9
    assert [int((r != 0).sum()) for r in q.float()] == [144, 0, 144, 0]
    assert bool((scale[[1, 3]] == 0).all()) and bool((scale[[0, 2]] > 0).all())


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(8, 16), (128, 128), (136, 144), (3, 264, 1040), (40, 72, 16), (2, 1536, 512)],
                         ids=str)
def test_quantize_weight(shape, dt, status):
    import pruned_expert_backward_gb300 as lrm
    g = gen(sum(shape))
    w = randn(g, *shape, dt=dt, std=0.05)
    w[..., 0, 3] = float("nan")
    w[..., -1, -1] = float("inf")
    for glu in (False, True):
        q, scale = lrm.lrm_fp8_quantize_weight(w, glu=glu)
        flat, per = w.view(-1, *shape[-2:]), 2 if glu else 1
        parts = [plain_blocks(h, 128) for e in flat for h in e.chunk(per)]
        same_bits(q, torch.cat([p[0].view(torch.uint8) for p in parts]).view(FP8).view(shape))
        same_bits(scale, torch.cat([p[1] for p in parts]).view(scale.shape))


# ------------------------------------------------------------------------------- products -------
def make(lrm, g, R, NP, K, E, act):
    x, xs = lrm.lrm_fp8_quantize(randn(g, R, K))
    lead = (E,) if E else ()
    w, ws = lrm.lrm_fp8_quantize_weight(randn(g, *lead, NP, K, std=K ** -0.5), glu=act == "swiglu")
    return x, xs, w, ws


DENSE = [  # R, N, K, act, bias, residual, save_z
    (1, 8, 16, "none", False, False, False), (1, 1408, 4096, "swiglu", True, False, False),
    (2, 72, 4112, "gelu", True, True, True), (5, 776, 64, "relu", False, True, False),
    (8, 4096, 1408, "none", True, True, False), (9, 136, 2048, "silu", True, True, True),
    (17, 264, 1040, "swiglu", False, True, True), (32, 520, 144, "silu", True, True, True),
    (33, 16, 32, "swiglu", True, True, True), (33, 256, 256, "gelu", True, False, True),
    (70, 8, 16, "gelu", True, True, True),
    (128, 256, 64, "swiglu", True, True, True), (129, 136, 80, "gelu", True, True, True),
    (257, 776, 1040, "swiglu", True, True, True), (300, 72, 2048, "relu", True, False, False),
    (1537, 776, 1040, "gelu", True, True, True), (3001, 1416, 528, "swiglu", True, False, True),
    (4096, 1024, 144, "silu", True, True, True), (4090, 512, 80, "swiglu", True, True, True),
    (2300, 136, 8208, "none", True, True, False),
    # tiles of 64, 128 and 256 columns, with a residual and without, SwiGLU and not (the rule of launch_fp8_tc)
    (300, 72, 272, "swiglu", True, False, True), (1000, 704, 144, "swiglu", True, True, True),
    (1000, 704, 400, "swiglu", False, False, True), (1500, 776, 144, "gelu", True, False, False),
    (4096, 1024, 272, "none", False, False, True), (4096, 512, 1168, "swiglu", False, False, False),
    (4001, 1000, 2064, "gelu", True, True, True),
]


@pytest.mark.parametrize("case", DENSE, ids=str)
def test_product(case, status):
    import pruned_expert_backward_gb300 as lrm
    R, N, K, act, bias, residual, save_z = case
    per = 2 if act == "swiglu" else 1
    g = gen(R + N)
    x, xs, w, ws = make(lrm, g, R, per * N, K, None, act)
    b = randn(g, per * N, std=0.3) if bias else None
    res = randn(g, R, N) if residual else None
    y, z = lrm.lrm_fp8_linear(x, xs, w, ws, bias=b, residual=res, act=act, save_z=save_z, dev_status=status)
    assert (z is not None) == save_z and y.dtype == BF16
    check_linear(operand(x, xs, 1), operand(w, ws, 128, per), b, res, act, None, y, z)


GROUPED = [  # R, E, segments, N, K, act, bias, residual, save_z
    (1, 4, "one", 64, 80, "swiglu", True, True, True), (8, 128, "ragged", 768, 256, "swiglu", False, False, False),
    (60, 5, "short", 136, 272, "gelu", True, True, True), (100, 5, "short", 136, 272, "gelu", True, True, True),
    (512, 128, "ragged", 264, 528, "swiglu", True, False, True), (512, 16, "one", 72, 144, "none", True, True, False),
    (1000, 3, "even", 520, 80, "silu", True, True, True), (2000, 7, "short", 264, 336, "swiglu", True, True, True),
    (5000, 40, "ragged", 392, 208, "relu", True, False, False), (3000, 1, "even", 136, 64, "swiglu", False, True, True),
    (6000, 1024, "ragged", 72, 64, "none", True, False, False),
    (3501, 5, "ragged", 1024, 144, "gelu", True, True, True),
    (3501, 5, "ragged", 1024, 400, "none", False, False, True),
    (3501, 5, "short", 512, 144, "swiglu", True, True, True), (9000, 2, "ragged", 136, 80, "gelu", True, True, True),
]


@pytest.mark.parametrize("case", GROUPED, ids=str)
def test_grouped_product(case, status):
    import pruned_expert_backward_gb300 as lrm
    R, E, kind, N, K, act, bias, residual, save_z = case
    per = 2 if act == "swiglu" else 1
    g = gen(R + E)
    seg = segments(kind, R, E, g)
    x, xs, w, ws = make(lrm, g, R, per * N, K, E, act)
    b = randn(g, E, per * N, std=0.3) if bias else None
    res = randn(g, R, N) if residual else None
    n = int(seg[-1])
    x.view(torch.uint8)[n:] = 0x7f  # rows of no expert are never used
    xs[n:] = float("nan")
    y = torch.full((R, N), 7.0, dtype=BF16, device="cuda")
    z = torch.full((R, per * N), 7.0, dtype=BF16, device="cuda") if save_z else None
    lrm.lrm_fp8_linear(x, xs, w, ws, bias=b, residual=res, act=act, seg_offsets=seg, y=y, z=z, dev_status=status)
    check_linear(operand(x, xs, 1), operand(w, ws, 128, per), b, res, act, seg, y, z)
    assert bool((y[n:] == 7.0).all()) and (z is None or bool((z[n:] == 7.0).all()))


GRADS = [  # R, E (None: dense), segments, N, K, glu
    (1, None, None, 16, 16, False), (1, None, None, 1408, 4096, True), (40, None, None, 128, 128, False),
    (257, None, None, 208, 1040, True), (1537, None, None, 784, 272, False), (3000, None, None, 136 + 8, 64, True),
    (512, 16, "one", 80, 144, True), (1222, 7, "short", 208, 1040, True), (3501, 5, "ragged", 512, 528, False),
    (6000, 1024, "ragged", 64, 80, True), (2000, 3, "even", 1536, 256, True),
]


@pytest.mark.parametrize("case", GRADS, ids=str)
def test_rows_gradient(case, status):
    import pruned_expert_backward_gb300 as lrm
    R, E, kind, N, K, glu = case
    per = 2 if glu else 1
    g = gen(R + N)
    seg = segments(kind, R, E, g) if E else None
    _, _, w, ws = make(lrm, g, 1, per * N, K, E, "swiglu" if glu else "none")
    dz, ds = lrm.lrm_fp8_quantize(randn(g, R, per * N, std=1e-3), glu=glu, dev_status=status)
    n = int(seg[-1]) if E else R
    dz.view(torch.uint8)[n:] = 0x7f
    ds[n:] = float("nan")
    dx = torch.full((R, K), 7.0, dtype=BF16, device="cuda")
    lrm.lrm_fp8_linear_backward(dz, ds, w, ws, glu=glu, seg_offsets=seg, dx=dx, dev_status=status)
    a, w64 = columns(dz, ds, per), operand(w, ws, 128, per).view(-1, per * N, K)
    for e, i, j in rows_of(seg, R):
        if j > i:
            check(dx[i:j], a[i:j] @ w64[e], (per * N + 1) * EPS * (a[i:j].abs() @ w64[e].abs()))
    assert bool((dx[n:] == 7.0).all())


def test_gradient_against_differences(status):
    """<dz, product(x + h) - product(x - h)> / 2 = <dx, h> for moves h that 8 bits hold exactly: the product without
    activation is linear in x, so the two sides differ by the roundings of y and dx alone."""
    import pruned_expert_backward_gb300 as lrm
    R, N, K, g = 300, 256, 384, gen(5)
    w, ws = lrm.lrm_fp8_quantize_weight(randn(g, N, K, std=K ** -0.5))
    one = torch.ones(R, 3, device="cuda")  # scales of 1: small integers are e4m3 values
    x = torch.randint(-3, 4, (R, K), generator=g, device="cuda").float()
    h = torch.randint(-2, 3, (R, K), generator=g, device="cuda").float()
    dz, ds = lrm.lrm_fp8_quantize(randn(g, R, N), dev_status=status)
    up, _ = lrm.lrm_fp8_linear((x + h).to(FP8), one, w, ws, dev_status=status)
    down, _ = lrm.lrm_fp8_linear((x - h).to(FP8), one, w, ws, dev_status=status)
    dx = lrm.lrm_fp8_linear_backward(dz, ds, w, ws, dev_status=status)
    d64 = operand(dz, ds, 1)
    left = (d64 * (up.double() - down.double())).sum(1) / 2
    right = (dx.double() * h.double()).sum(1)
    ends = (d64.abs() * (up.abs() + down.abs()).double()).sum(1) / 2
    slack = 2.0 ** -8 * (ends + (dx.abs() * h.abs()).double().sum(1))
    assert bool(((left - right).abs() <= slack).all())


@pytest.mark.parametrize("R", [3, 300])
def test_nan_stays_in_its_row_and_column(R, status):
    import pruned_expert_backward_gb300 as lrm
    N, K, g = 272, 400, gen(R)
    x0, w0 = randn(g, R, K), randn(g, N, K, std=0.05)
    x0[1, 140] = float("nan")
    w0[200, 399] = float("inf")  # its block is rows 128 to 255
    x, xs = lrm.lrm_fp8_quantize(x0, dev_status=status)
    w, ws = lrm.lrm_fp8_quantize_weight(w0)
    y, _ = lrm.lrm_fp8_linear(x, xs, w, ws, dev_status=status)
    bad = torch.isnan(y)
    assert bool(bad[1].all()) and bool(bad[:, 128:256].all())
    bad[1], bad[:, 128:256] = False, False
    assert not bool(bad.any())


@pytest.mark.parametrize("act", ["gelu", "silu", "swiglu", "relu"])
def test_large_pre_activations(act, status):
    """Saturated activations: |z| up to 1e4 gives 0, z or the product, never NaN."""
    import pruned_expert_backward_gb300 as lrm
    per = 2 if act == "swiglu" else 1
    for R in (4, 200):
        g = gen(R)
        x, xs = lrm.lrm_fp8_quantize(randn(g, R, 256, std=30.0), dev_status=status)
        w, ws = lrm.lrm_fp8_quantize_weight(randn(g, per * 64, 256, std=10.0), glu=act == "swiglu")
        y, z = lrm.lrm_fp8_linear(x, xs, w, ws, act=act, save_z=True, dev_status=status)
        assert bool(torch.isfinite(y).all())
        check_linear(operand(x, xs, 1), operand(w, ws, 128, per), None, None, act, None, y, z)


def test_bad_segments_compute_nothing():
    import pruned_expert_backward_gb300 as lrm
    g = gen(2)
    for R in (20, 200):
        x, xs, w, ws = make(lrm, g, R, 64, 64, 3, "none")
        dz, ds = lrm.lrm_fp8_quantize(randn(g, R, 64))
        for bad in ([1, 5, 9, R], [0, 9, 5, R], [0, 5, 9, R + 1], [0, -1, 9, R]):
            seg = torch.tensor(bad, dtype=torch.int32, device="cuda")
            for call in ("forward", "backward"):
                st = torch.zeros(1, dtype=torch.int32, device="cuda")
                out = torch.full((R, 64), 7.0, dtype=BF16, device="cuda")
                if call == "forward":
                    lrm.lrm_fp8_linear(x, xs, w, ws, seg_offsets=seg, y=out, dev_status=st)
                else:
                    lrm.lrm_fp8_linear_backward(dz, ds, w, ws, seg_offsets=seg, dx=out, dev_status=st)
                assert int(st.item()) == 11 and bool((out == 7.0).all())


def test_no_rows(status):
    import pruned_expert_backward_gb300 as lrm
    x, xs = lrm.lrm_fp8_quantize(torch.zeros(0, 64, dtype=BF16, device="cuda"), dev_status=status)
    assert tuple(x.shape) == (0, 64) and tuple(xs.shape) == (0, 1)
    w, ws = lrm.lrm_fp8_quantize_weight(torch.ones(32, 64, dtype=BF16, device="cuda"))
    y, _ = lrm.lrm_fp8_linear(x, xs, w, ws, dev_status=status)
    dx = lrm.lrm_fp8_linear_backward(torch.zeros(0, 32, device="cuda").to(FP8), torch.zeros(0, 1, device="cuda"), w, ws)
    assert tuple(y.shape) == (0, 32) and tuple(dx.shape) == (0, 64)
    seg = torch.zeros(4, dtype=torch.int32, device="cuda")  # rows there, but of no expert
    for R in (5, 500):
        x, xs, w3, ws3 = make(lrm, gen(1), R, 32, 64, 3, "none")
        y = torch.full((R, 32), 7.0, dtype=BF16, device="cuda")
        lrm.lrm_fp8_linear(x, xs, w3, ws3, seg_offsets=seg, y=y, dev_status=status)
        assert bool((y == 7.0).all())


def test_same_bits_again_on_another_stream_and_in_a_graph(status):
    import pruned_expert_backward_gb300 as lrm
    R, E, g = 700, 5, gen(3)
    seg = segments("ragged", R, E, g)
    x0 = randn(g, R, 272)
    _, _, w, ws = make(lrm, g, 1, 2 * 136, 272, E, "swiglu")
    dz0 = randn(g, R, 2 * 144)
    _, _, w2, ws2 = make(lrm, g, 1, 2 * 144, 272, E, "swiglu")

    def step():
        x, xs = lrm.lrm_fp8_quantize(x0, dev_status=status)
        y, z = lrm.lrm_fp8_linear(x, xs, w, ws, act="swiglu", seg_offsets=seg, save_z=True, dev_status=status)
        dz, ds = lrm.lrm_fp8_quantize(dz0, glu=True, dev_status=status)
        return y, z, lrm.lrm_fp8_linear_backward(dz, ds, w2, ws2, glu=True, seg_offsets=seg, dev_status=status)

    n = int(seg[-1])
    first = [t[:n].clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, other, kept):
        assert torch.equal(a, b[:n]) and torch.equal(a, c[:n])
    x0.neg_()  # the graph reads the inputs that are there
    graph.replay()
    again = step()
    torch.cuda.synchronize()
    assert all(torch.equal(b[:n], c[:n]) for b, c in zip(again, kept)) and not torch.equal(kept[0][:n], first[0])


def test_refusals():
    import pruned_expert_backward_gb300 as lrm
    x = torch.zeros(40, 64, dtype=BF16, device="cuda")
    q, s = lrm.lrm_fp8_quantize(x)
    w, ws = lrm.lrm_fp8_quantize_weight(torch.zeros(32, 64, dtype=BF16, device="cuda"))
    for call in (lambda: lrm.lrm_fp8_quantize(x.cpu()), lambda: lrm.lrm_fp8_quantize(x.t()),
                 lambda: lrm.lrm_fp8_quantize(x, k=2), lambda: lrm.lrm_fp8_quantize(x, q=q[:20]),
                 lambda: lrm.lrm_fp8_quantize(x, row_of_pair=torch.zeros(7, dtype=torch.int32, device="cuda"), k=2),
                 lambda: lrm.lrm_fp8_quantize_weight(x.view(-1)), lambda: lrm.lrm_fp8_linear(q, s[:5], w, ws),
                 lambda: lrm.lrm_fp8_linear(q, s, w, ws[:, :0]), lambda: lrm.lrm_fp8_linear(q[:, :32], s, w, ws),
                 lambda: lrm.lrm_fp8_linear(q, s, w, ws, bias=x[0]),
                 lambda: lrm.lrm_fp8_linear(q, s, w, ws, act="tanh"),
                 lambda: lrm.lrm_fp8_linear(q, s, w, ws, residual=x), lambda: lrm.lrm_fp8_linear_backward(q, s, w, ws)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lrm.lrm_fp8_quantize(x.half()), lambda: lrm.lrm_fp8_linear(x, s, w, ws),
                 lambda: lrm.lrm_fp8_linear(q, s, x[:32], ws), lambda: lrm.lrm_fp8_linear(q, s.double(), w, ws)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(lrm.LrmError):
        lrm.lrm_fp8_quantize(torch.zeros(4, 72, dtype=BF16, device="cuda"))  # rows off the 16 bytes
