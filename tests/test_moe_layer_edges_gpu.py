"""GPU checks of the MoE layer's entry points at their limits, against 64-bit plain forms.

Tolerances as in test_moe_layer_gpu.py, whose checks are used here."""
import pytest
import torch

from helpers import ensure_built
from test_moe_layer_gpu import BF16, F32, gen, randn

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
