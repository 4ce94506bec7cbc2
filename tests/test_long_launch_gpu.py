"""Launches of more than a second: the bound on the tile kernels' waits counts what a wait stands for, not the launch."""
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu


def test_a_product_of_more_than_a_second():
    """fp32, 65536 x 65536 x 65536: six bf16 products of 5.6e14 operations each, 1.7 s at 2 PFLOP/s.  One CTA of each
    pair waits through all of it for the other's last products.  Tolerance: sums of 65536 products in fp32 err by
    65537 * 2^-23 of the sum of magnitudes at most."""
    import pruned_expert_backward_gb300 as lrm
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()
    n = 65536
    if torch.cuda.mem_get_info()[0] < 150e9:
        pytest.skip("needs 150 GB")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, w = (torch.randn(n, n, generator=g, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, _ = lrm.lrm_linear(x, w, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    at = torch.tensor([0, 127, 128, 255, 256, 20000, 40129, n - 129, n - 128, n - 1], device="cuda")
    for rows, cols in ((at, slice(None, None, 61)), (slice(None, None, 61), at)):
        a, b = x[rows].double(), w[cols].double()
        slack = (n + 1) * 2.0 ** -23 * (a.abs() @ b.abs().t())
        assert bool(((y[rows][:, cols].double() - a @ b.t()).abs() <= slack).all())
