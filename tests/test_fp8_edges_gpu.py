"""Edges of the 8-bit operators: infinite and NaN pre-activations, whichever kernel a call takes."""
import pytest
import torch

from helpers import ensure_built
from test_fp8_gpu import BF16, F32, operand, plain_blocks, same_bits, status  # noqa: F401
from test_moe_layer_gpu import check_linear, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def act64(z, act):
    if act == "swiglu":
        gate, up = z.chunk(2, 1)
        return gate * torch.special.expit(gate) * up
    return {"none": lambda v: v, "relu": lambda v: torch.where(v < 0, torch.zeros_like(v), v),
            "gelu": lambda v: v * torch.special.ndtr(v), "silu": lambda v: v * torch.special.expit(v)}[act](z)


@pytest.mark.parametrize("residual", [False, True], ids=["", "residual"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("R", [4, 16, 40, 200, 3000])
def test_infinite_pre_activations(R, act, residual, status):  # noqa: F811
    """+inf, -inf and NaN by the bias: the outputs' kinds are the 64-bit formula's for any number of rows (0 * inf is
    NaN there too), their neighbours are as ever."""
    import pruned_expert_backward_gb300 as lrm
    per, N, K, g = 2 if act == "swiglu" else 1, 520, 144, gen(R)
    x, xs = lrm.lrm_fp8_quantize(randn(g, R, K), dev_status=status)
    w, ws = lrm.lrm_fp8_quantize_weight(randn(g, per * N, K, std=K ** -0.5), glu=act == "swiglu")
    b = randn(g, per * N, std=0.3)
    inf, nan = float("inf"), float("nan")
    b[3], b[40], b[77], b[300] = inf, -inf, nan, inf
    if per == 2:
        b[N + 3], b[N + 40], b[N + 100], b[N + 101] = -inf, inf, inf, nan
    res = randn(g, R, N) if residual else None
    y, z = lrm.lrm_fp8_linear(x, xs, w, ws, bias=b, residual=res, act=act, save_z=True, dev_status=status)
    z64 = operand(x, xs, 1) @ operand(w, ws, 128, per).t() + b.double()
    want = act64(z64, act) + (res.double() if residual else 0)
    for got, ref in ((z, z64), (y, want)):
        got = got.double()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.isposinf(got), torch.isposinf(ref))
        assert torch.equal(torch.isneginf(got), torch.isneginf(ref))
    usual = torch.isfinite(b.view(per, N)).all(0)
    cols = torch.nonzero(usual).flatten()
    rows = torch.cat([cols + i * N for i in range(per)])
    # (a column's operand does not depend on its neighbours: the usual columns, checked as a product of their own)
    check_linear(operand(x, xs, 1), operand(w, ws, 128, per)[rows], b[rows], res[:, cols] if residual else None, act,
                 None, y[:, cols], z[:, rows])


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("R", [4, 300, 2000])
def test_residual_in_place(R, act, status):  # noqa: F811
    """y and the residual the same tensor: each output's residual is read before it is written."""
    import pruned_expert_backward_gb300 as lrm
    per, K = 2 if act == "swiglu" else 1, 272
    for N in (520, 528):  # rows off and on the 32-byte sectors
        g = gen(R + N)
        x, xs = lrm.lrm_fp8_quantize(randn(g, R, K), dev_status=status)
        w, ws = lrm.lrm_fp8_quantize_weight(randn(g, per * N, K, std=K ** -0.5), glu=act == "swiglu")
        res = randn(g, R, N)
        y, _ = lrm.lrm_fp8_linear(x, xs, w, ws, residual=res, act=act, dev_status=status)
        same = res.clone()
        got, _ = lrm.lrm_fp8_linear(x, xs, w, ws, residual=same, act=act, y=same, dev_status=status)
        assert got is same and torch.equal(same, y)
        check_linear(operand(x, xs, 1), operand(w, ws, 128, per), None, res, act, None, y, None)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 32), (5, 288), (130, 4128), (33, 416)], ids=str)
def test_quantize_halves(shape, dt, status):  # noqa: F811
    """SwiGLU's gradient: gate and up columns in blocks of their own."""
    import pruned_expert_backward_gb300 as lrm
    x = randn(gen(sum(shape)), *shape, dt=dt, std=1e-3)
    x[0, 1], x[-1, -1] = 7.0, float("nan")
    q, scale = lrm.lrm_fp8_quantize(x, glu=True, dev_status=status)
    parts = [plain_blocks(h, 1) for h in x.chunk(2, 1)]
    same_bits(q, torch.cat([p[0].float() for p in parts], 1))
    same_bits(scale, torch.cat([p[1] for p in parts], 1))


def test_outputs_past_31_bits(status):  # noqa: F811
    """Products and row gradients whose outputs hold more than 2^31 values: the rows at the ends and about 2^31."""
    import pruned_expert_backward_gb300 as lrm
    N, K = 2048, 32
    R = (1 << 31) // N + 3001
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 30 GB")
    g = gen(9)
    near = [0, 300, (1 << 31) // N - 130, (1 << 31) // N, (1 << 31) // N + 129, R - 300]
    at = torch.cat([torch.arange(a, a + 128, device="cuda") for a in near] + [torch.arange(R - 1, R, device="cuda")])
    x, xs = lrm.lrm_fp8_quantize(randn(g, R, K), dev_status=status)
    w, ws = lrm.lrm_fp8_quantize_weight(randn(g, N, K, std=K ** -0.5))
    res = randn(g, 1, N).expand(R, N).contiguous()
    for residual in (None, res):
        y, _ = lrm.lrm_fp8_linear(x, xs, w, ws, residual=residual, dev_status=status)
        check_linear(operand(x[at], xs[at], 1), operand(w, ws, 128), None, None if residual is None else residual[at],
                     "none", None, y[at], None)
        del y
    del res
    dz, ds = lrm.lrm_fp8_quantize(randn(g, R, K), dev_status=status)
    w2, ws2 = lrm.lrm_fp8_quantize_weight(randn(g, K, N, std=K ** -0.5))
    dx = lrm.lrm_fp8_linear_backward(dz, ds, w2, ws2, dev_status=status)
    check_linear(operand(dz[at], ds[at], 1), operand(w2, ws2, 128).t(), None, None, "none", None, dx[at], None)
