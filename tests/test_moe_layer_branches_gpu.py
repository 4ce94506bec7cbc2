"""GPU parity of the products' kernels that test_moe_layer_gpu.py's sizes do not choose: 256-column tiles in every
type, whole and in parts, dense and per expert, operands in one box, and the one-pass kernel over its whole range.

Which kernel a size takes follows the rules of cut_product, with_width, cut_rows and linear_few_rows for the 76 CTA
pairs of a GB300.  Tolerances as in test_moe_layer_gpu.py, whose checks are used here."""
import pytest
import torch

from helpers import ensure_built
from test_moe_layer_gpu import BF16, EPS, F32, check, check_linear, gen, linear_inputs, randn, rows_of, segments

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


PRODUCTS = [  # dtype, R, E (None: dense), segments, N, K, act, fp32 output, bias, residual, save_z
    # 256-column tiles
    (BF16, 4096, None, None, 1024, 144, "gelu", False, True, True, True),
    (BF16, 4096, None, None, 1024, 136, "gelu", False, True, True, True),  # weights copied to aligned rows
    (BF16, 3501, 5, "ragged", 1024, 144, "relu", False, True, True, True),
    (BF16, 3501, 5, "short", 512, 144, "swiglu", False, True, True, True),
    (BF16, 4096, None, None, 1024, 144, "silu", True, True, False, True),
    (BF16, 3501, 5, "ragged", 1016, 144, "none", True, True, False, True),
    (BF16, 4090, None, None, 512, 80, "swiglu", True, True, False, True),
    (BF16, 3501, 5, "short", 512, 72, "swiglu", True, False, False, True),
    (F32, 4090, None, None, 1024, 136, "gelu", False, True, True, True),
    (F32, 3501, 5, "ragged", 1024, 136, "relu", False, True, True, True),
    (F32, 4096, None, None, 512, 72, "swiglu", False, True, True, True),
    (F32, 3501, 5, "short", 504, 136, "swiglu", False, True, True, True),
    # 128 columns
    (BF16, 1537, None, None, 776, 136, "gelu", True, True, False, True),
    (BF16, 1500, 5, "ragged", 776, 136, "silu", True, True, False, True),
    (BF16, 700, None, None, 136, 136, "swiglu", True, True, False, True),
    (BF16, 700, 5, "short", 136, 136, "swiglu", True, True, False, True),
    (F32, 1537, None, None, 776, 136, "silu", False, True, True, True),
    (F32, 1500, 5, "short", 776, 136, "silu", False, True, True, True),
    (BF16, 1300, 9, "ragged", 136, 264, "gelu", True, True, False, True),  # 64
    # long sums of bf16 results
    (BF16, 4096, None, None, 1024, 65544, "gelu", False, True, True, True),
    (BF16, 4096, None, None, 512, 65552, "swiglu", False, True, True, True),
    (BF16, 1100, 3, "ragged", 512, 65544, "none", False, True, True, False),
    # sums in parts: 256, 128 and 64 columns
    (F32, 2300, None, None, 512, 1024, "gelu", False, True, True, True),
    (F32, 2300, None, None, 264, 1024, "swiglu", False, True, True, True),
    (F32, 2100, 2, "ragged", 512, 1200, "relu", False, True, True, True),
    (F32, 2100, 2, "short", 256, 1200, "swiglu", False, True, True, True),
    (BF16, 1000, 2, "ragged", 1000, 12000, "gelu", True, True, False, True),
    (BF16, 100, None, None, 264, 9000, "swiglu", False, True, True, True),
    (BF16, 64, None, None, 1408, 16384, "swiglu", False, True, True, True),
    (BF16, 200, 3, "ragged", 264, 6000, "gelu", False, True, True, True),
    (BF16, 200, 3, "short", 136, 8192, "swiglu", False, True, True, True),
    (BF16, 1000, None, None, 1024, 12000, "none", False, True, True, True),
    (BF16, 300, 4, "one", 136, 8192, "none", True, True, False, True),
    # one pass over the weights: dense
    (F32, 5, None, None, 136, 264, "gelu", False, True, True, True),
    (F32, 8, None, None, 72, 1032, "swiglu", False, True, True, True),
    (F32, 9, None, None, 136, 264, "swiglu", False, True, True, True),
    (F32, 17, None, None, 264, 520, "silu", False, True, True, True),
    (F32, 24, None, None, 72, 2056, "none", False, True, True, True),
    (BF16, 12, None, None, 264, 520, "swiglu", False, True, True, True),
    (BF16, 24, None, None, 264, 1032, "gelu", False, True, True, True),
    (BF16, 32, None, None, 136, 2056, "none", False, True, True, True),
    (BF16, 7, None, None, 128, 4096, "none", True, True, False, True),
    (BF16, 32, None, None, 128, 4096, "silu", True, True, False, True),
    (BF16, 5, None, None, 72, 264, "swiglu", True, True, False, True),
    (BF16, 15, None, None, 72, 264, "swiglu", True, True, False, True),
    (BF16, 31, None, None, 72, 264, "swiglu", True, True, False, True),
    # per expert
    (BF16, 40, 6, "one", 136, 264, "gelu", False, True, True, True),
    (BF16, 64, 6, "one", 72, 520, "swiglu", False, True, True, True),
    (BF16, 64, 40, "ragged", 264, 136, "none", False, True, True, True),
    (BF16, 50, 3, "short", 136, 264, "swiglu", False, True, True, True),
    (BF16, 29, 12, "ragged", 128, 1032, "relu", True, True, False, True),
    (BF16, 61, 4, "even", 72, 136, "swiglu", True, True, False, True),
    (F32, 8, 128, "ragged", 72, 136, "swiglu", False, True, True, True),
    (F32, 32, 2, "even", 136, 264, "gelu", False, True, True, True),
    (F32, 64, 16, "ragged", 136, 264, "swiglu", False, True, True, True),
    (F32, 300, 64, "one", 72, 520, "silu", False, True, True, True),
    (F32, 512, 64, "ragged", 264, 136, "none", False, True, True, True),
    (F32, 8000, 1000, "ragged", 40, 72, "swiglu", False, True, True, True),
    (F32, 72, 9, "short", 40, 1032, "relu", False, False, True, True),
]


@pytest.mark.parametrize("case", PRODUCTS, ids=str)
def test_products(case, status):
    import pruned_expert_backward_gb300 as lrm
    dt, R, E, kind, N, K, act, out_f32, bias, residual, save_z = case
    NP = 2 * N if act == "swiglu" else N
    g = gen(R + N)
    seg = segments(kind, R, E, g) if E else None
    x, w, b, res = linear_inputs(g, dt, R, NP, N, K, bias, residual, E)
    n = int(seg[-1]) if E else R
    x[n:] = float("nan")  # rows of no expert are never used
    y = torch.full((R, N), 7.0, dtype=F32 if out_f32 else dt, device="cuda")
    z = torch.full((R, NP), 7.0, dtype=dt, device="cuda") if save_z else None
    lrm.lrm_linear(x, w, bias=b, residual=res, act=act, seg_offsets=seg, y=y, z=z, dev_status=status)
    check_linear(x, w, b, res, act, seg, y, z)
    assert bool((y[n:] == 7.0).all()) and (z is None or bool((z[n:] == 7.0).all()))


GRADIENTS = [  # dtype, R, E (None: dense), segments, N, K
    # dW in 256-column tiles, operands in one box or not, whole and in runs of rows
    (BF16, 300, None, None, 1024, 4096), (F32, 300, None, None, 1024, 4096), (F32, 300, None, None, 1032, 4104),
    (BF16, 3000, 8, "ragged", 512, 1024), (F32, 3000, 8, "short", 512, 1024), (BF16, 3000, 8, "short", 512, 1000),
    (BF16, 3000, 8, "one", 504, 1024), (BF16, 30000, 3, "ragged", 128, 512), (F32, 9000, 6, "short", 128, 512),
    # dx in 256-column tiles
    (BF16, 4096, None, None, 136, 1024), (BF16, 4090, None, None, 136, 1000), (F32, 4096, None, None, 136, 1024),
    (BF16, 3501, 5, "ragged", 136, 1024), (F32, 3501, 5, "short", 136, 1024), (F32, 4096, None, None, 72, 1000),
    # dx in parts: 256 and 128 columns
    (F32, 2300, None, None, 1024, 512), (F32, 2100, 2, "ragged", 1200, 512), (BF16, 1000, None, None, 12000, 1024),
    (BF16, 900, None, None, 12000, 1000), (BF16, 1000, 2, "short", 12000, 1000), (BF16, 300, None, None, 8200, 72),
    (BF16, 200, 4, "short", 8200, 136),
    # long sums of bf16 results
    (BF16, 10240, None, None, 65544, 128),
]


@pytest.mark.parametrize("case", GRADIENTS, ids=str)
def test_gradients(case, status):
    import pruned_expert_backward_gb300 as lrm
    dt, R, E, kind, N, K = case
    g = gen(R + N + K)
    seg = segments(kind, R, E, g) if E else None
    x, w, _, _ = linear_inputs(g, dt, R, N, N, K, False, False, E)
    dz = randn(g, R, N, dt=dt)
    n = int(seg[-1]) if E else R
    x[n:], dz[n:] = float("nan"), float("nan")
    dx = torch.full((R, K), 7.0, dtype=dt, device="cuda")
    _, dw = lrm.lrm_linear_backward(dz, x, w, seg_offsets=seg, dx=dx, dev_status=status)
    assert bool((dx[n:] == 7.0).all())
    for e, a, b in rows_of(seg, R):
        we, xe, de = w.view(-1, N, K)[e].double(), x[a:b].double(), dz[a:b].double()
        check(dx[a:b], de @ we, (N + 1) * EPS * (de.abs() @ we.abs()))
        got, want = dw.view(-1, N, K)[e], de.t() @ xe
        if a == b:
            assert torch.count_nonzero(got) == 0
            continue
        check(got, want, (b - a + 1) * EPS * (de.abs().t() @ xe.abs()))
        assert (got.double() - want).norm() <= 5e-6 * want.norm()


# ------------------------------------------------------------------------------- debug build ----
_EVERY_CALL = r"""
import os, sys, torch
sys.path.insert(0, sys.argv[1]); sys.path.insert(0, sys.argv[1] + "/tests")
from pruned_expert_backward_gb300 import _lib
assert _lib.library_path().endswith(sys.argv[3])
import pruned_expert_backward_gb300 as lrm
from test_moe_layer_gpu import BF16, F32, gen, linear_inputs, randn, routing, segments
st, out = torch.zeros(1, dtype=torch.int32, device="cuda"), []
for T, k, E, H, dt in ((3, 8, 16, 520, BF16), (40, 4, 300, 72, F32), (700, 8, 60, 512, BF16), (3000, 6, 60, 136, F32),
                       (2000, 1, 7, 1032, BF16)):
    g = gen(T)
    idx, alpha = routing(g, T, k, E, 1.0, 0.2)
    seg, pair, row, x_s = lrm.lrm_sort_tokens(idx, randn(g, T, H, dt=dt), E, dev_status=st)
    out += [seg, pair, row, x_s, lrm.lrm_combine(row, alpha, x_s, dev_status=st)]
    out += lrm.lrm_combine_backward(row, alpha, randn(g, T, H, dt=dt), x_s, dy_s=torch.zeros_like(x_s), dev_status=st)
sizes = [(3, None, 72, 136), (8, 16, 72, 136), (300, None, 136, 264), (900, 7, 136, 264), (4096, None, 1024, 72),
         (12000, 3, 128, 264), (200, 3, 72, 4096), (50, None, 72, 4096), (150, 2, 4104, 72)]
for R, E, N, K in sizes:
    for dt in (BF16, F32):
        for simt in (0, 1):
            g = gen(R)
            seg = segments("short", R, E, g) if E else None
            x, w, b, res = linear_inputs(g, dt, R, 2 * N, N, K, True, True, E)
            y, z, dz = torch.zeros_like(res), randn(g, R, 2 * N, dt=dt), torch.zeros(R, 2 * N, dtype=dt, device="cuda")
            lrm.lrm_linear(x, w, bias=b, residual=res, act="swiglu", seg_offsets=seg, y=y, flags=simt, dev_status=st)
            _, db = lrm.lrm_act_backward(res, z, act="swiglu", seg_offsets=seg, dz=dz, dev_status=st)
            dx = torch.zeros_like(x)
            _, dw = lrm.lrm_linear_backward(dz, x, w, seg_offsets=seg, dx=dx, flags=simt, dev_status=st)
            out += [y, dz, db, dx, dw]
assert int(st.item()) == 0, int(st.item())
torch.save([t.cpu() for t in out], sys.argv[2])
"""


def test_debug_build_checks_the_layer_and_matches_release(tmp_path):
    """liblrm_debug.so runs every call of the layer with no index check failing, and gives the same bits."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    results = []
    for debug, name in (("1", "liblrm_debug.so"), ("0", "liblrm.so")):
        path = str(tmp_path / name) + ".pt"
        r = subprocess.run([sys.executable, "-c", _EVERY_CALL, root, path, "/" + name],
                           env=dict(os.environ, LRM_DEBUG=debug), capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout + r.stderr
        results.append(torch.load(path))
    assert len(results[0]) == len(results[1]) > 100
    for a, b in zip(*results):
        assert torch.equal(a, b)
