"""The MoE layer in 8 bits with its optimiser, run together as they would be used.

Each call of the layer is checked against the 64-bit form of the operands it was given (the tolerances of
test_fp8_gpu.py and test_moe_layer_gpu.py), which holds the whole to the sum of its parts; against the bf16 layer the
whole stays within what the operands' rounding gives: 0.036 of each operand at most (2^-4 / 3^0.5), so 0.051 of a
product, 0.08 after SwiGLU (two of them and their slopes), 0.1 after the second product.  0.15 is allowed.
"""
import os
import subprocess
import sys

import pytest
import torch

from helpers import ensure_built
from test_fp8_gpu import columns, operand, same_bits
from test_moe_layer_gpu import EPS, check, check_linear, gen, randn, rows_of, routing

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def make(T, k, E, H, I, masked=0.0):
    g = gen(T + E)
    idx, alpha = routing(g, T, k, E, 1.0, masked)
    return (randn(g, T, H), randn(g, T, H, std=1e-2), idx, alpha, randn(g, E, 2 * I, H, std=H ** -0.5),
            randn(g, E, H, I, std=I ** -0.5))


SIZES = [(1, 2, 4, 64, 32, 0.0), (40, 4, 16, 272, 144, 0.2), (700, 8, 60, 512, 208, 0.1), (2000, 2, 5, 1024, 384, 0.0)]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_layer(size):
    import pruned_expert_backward_gb300 as lrm
    T, k, E, H, I, masked = size
    x, dy, idx, alpha, w1, w2 = make(*size)
    q1, q2 = lrm.lrm_fp8_quantize_weight(w1, glu=True), lrm.lrm_fp8_quantize_weight(w2)
    layer = lrm.MoeLayer(T, k, E, H, I, fp8=True)
    y = layer.forward(x, idx, alpha, q1, q2, residual=x).clone()
    seg = layer.seg_offsets
    n = int(seg[-1])
    v1, v2 = operand(*q1, 128, 2), operand(*q2, 128)
    check_linear(operand(*layer.xq, 1)[:n], v1, None, None, "swiglu", seg, layer.phi_s[:n], layer.h_s[:n])
    check_linear(operand(*layer.phiq, 1)[:n], v2, None, None, "none", seg, layer.y_s[:n], None)
    dx, dalpha, dw1, dw2 = [t.clone() for t in layer.backward(dy, alpha, q1, q2)]
    assert int(layer.dev_status.item()) == 0
    a1, a2 = columns(*layer.dhq, 2), operand(*layer.dyq, 1)
    for e, i, j in rows_of(seg, n):
        if i == j:
            assert torch.count_nonzero(dw1[e]) == 0 and torch.count_nonzero(dw2[e]) == 0
            continue
        check(layer.dphi_s[i:j], a2[i:j] @ v2[e], (H + 1) * EPS * (a2[i:j].abs() @ v2[e].abs()))
        check(layer.dx_s[i:j], a1[i:j] @ v1[e], (2 * I + 1) * EPS * (a1[i:j].abs() @ v1[e].abs()))
        for dw, d, rows in ((dw1, layer.dh_s, layer.x_s), (dw2, layer.dy_s, layer.phi_s)):
            d, rows = d[i:j].double(), rows[i:j].double()
            check(dw[e], d.t() @ rows, (j - i + 1) * EPS * (d.abs().t() @ rows.abs()))
    # against the layer in bf16, and served as trained
    full = lrm.MoeLayer(T, k, E, H, I)
    near = full.forward(x, idx, alpha, w1, w2, residual=x)

    def far(a, b):
        return ((a.double() - b.double()).norm() / b.double().norm().clamp_min(1e-30)).item()

    assert far(y.double() - x.double(), near.double() - x.double()) <= 0.15
    dx_full, _, dw1_full, dw2_full = full.backward(dy, alpha, w1, w2)
    for a, b in ((dx, dx_full), (dw1, dw1_full), (dw2, dw2_full)):
        assert far(a, b) <= 0.2  # (one more product in the chain)
    served = lrm.MoeLayer(T, k, E, H, I, fp8=True, train=False)
    assert torch.equal(served.forward(x, idx, alpha, q1, q2, residual=x), y)
    with pytest.raises(ValueError):
        served.backward(dy, alpha, q1, q2)


def test_training_steps_with_the_optimiser():
    """Forward, backward, AdamW with 8-bit states on the layer's gradients, weights to 8 bits again; then the same two
    steps from a captured graph."""
    import pruned_expert_backward_gb300 as lrm
    T, k, E, H, I = 300, 4, 8, 256, 128
    results = []
    for captured in (False, True):
        x, dy, idx, alpha, w1, w2 = make(T, k, E, H, I)
        q1, q2 = lrm.lrm_fp8_quantize_weight(w1, glu=True), lrm.lrm_fp8_quantize_weight(w2)
        layer = lrm.MoeLayer(T, k, E, H, I, fp8=True)
        opt = lrm.AdamW([w1, w2], [layer.dw_gate_up, layer.dw_down], lr=1e-3, betas=(0.9, 0.95), weight_decay=0.1,
                        state_bits=8, max_norm=1.0, seed=3, capturable=True)

        def step():
            layer.forward(x, idx, alpha, q1, q2)
            layer.backward(dy, alpha, q1, q2)
            opt.step()
            lrm.lrm_fp8_quantize_weight(w1, glu=True, q=q1[0], scale=q1[1])
            lrm.lrm_fp8_quantize_weight(w2, q=q2[0], scale=q2[1])

        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for _ in range(2):
            before = [w1.clone(), w2.clone(), *[s.clone() for s in opt.state["m"]]]
            graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert int(layer.dev_status.item()) == 0 and int(opt.dev_status.item()) == 0
        same_bits(q1[0], lrm.lrm_fp8_quantize_weight(w1, glu=True)[0])
        norm = (layer.dw_gate_up.double().square().sum() + layer.dw_down.double().square().sum()).sqrt().item()
        assert abs(opt.norm.item() / norm - 1) < 1e-6
        for new, old in zip((w1, w2, *opt.state["m"]), before):
            assert not torch.equal(new.view(torch.uint8), old.view(torch.uint8))
        results.append([w1.clone(), w2.clone(), q1[1].clone(), layer.y.clone(), layer.dx.clone()])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_layer_takes_no_memory_after_the_first_call():
    import pruned_expert_backward_gb300 as lrm
    T, k, E, H, I = 3000, 4, 12, 256, 128
    x, dy, idx, alpha, w1, w2 = make(T, k, E, H, I, 0.1)
    q1, q2 = lrm.lrm_fp8_quantize_weight(w1, glu=True), lrm.lrm_fp8_quantize_weight(w2)
    layer, served = lrm.MoeLayer(T, k, E, H, I, fp8=True), lrm.MoeLayer(T, k, E, H, I, fp8=True, train=False)
    opt = lrm.AdamW([w1, w2], [layer.dw_gate_up, layer.dw_down], state_bits=8, max_norm=1.0)

    def step():
        layer.forward(x, idx, alpha, q1, q2, residual=x)
        layer.backward(dy, alpha, q1, q2)
        opt.step()
        lrm.lrm_fp8_quantize_weight(w1, glu=True, q=q1[0], scale=q1[1])
        served.forward(x, idx, alpha, q1, q2)

    step()
    torch.cuda.synchronize()
    made, free = torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]
    step()
    torch.cuda.synchronize()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == made
    assert torch.cuda.mem_get_info()[0] == free


def test_layer_without_tokens_and_refusals():
    import pruned_expert_backward_gb300 as lrm
    x, dy, idx, alpha, w1, w2 = make(4, 2, 4, 64, 32)
    q1, q2 = lrm.lrm_fp8_quantize_weight(w1, glu=True), lrm.lrm_fp8_quantize_weight(w2)
    layer = lrm.MoeLayer(0, 2, 4, 64, 32, fp8=True)
    y = layer.forward(x[:0], idx[:0], alpha[:0], q1, q2)
    dx, dalpha, dw1, dw2 = layer.backward(dy[:0], alpha[:0], q1, q2)
    assert tuple(y.shape) == (0, 64) and torch.count_nonzero(dw1) == 0 and torch.count_nonzero(dw2) == 0
    layer = lrm.MoeLayer(4, 2, 4, 64, 32, fp8=True)
    idx[:] = -1  # no pair is routed
    y = layer.forward(x, idx, alpha, q1, q2, residual=x)
    assert torch.equal(y, x)
    dx, dalpha, dw1, dw2 = layer.backward(dy, alpha, q1, q2)
    assert all(torch.count_nonzero(t) == 0 for t in (dx, dalpha, dw1, dw2))
    assert int(layer.dev_status.item()) == 0
    for kw in (dict(dtype=torch.float32), dict(flags=1)):
        with pytest.raises(ValueError):
            lrm.MoeLayer(4, 2, 4, 64, 32, fp8=True, **kw)
    with pytest.raises(ValueError):
        lrm.MoeLayer(4, 2, 4, 72, 32, fp8=True)
    with pytest.raises(ValueError):
        lrm.lrm_linear_backward(dy, x, None)
    for other, a, b in ((layer, w1, w2), (layer, q1, w2), (lrm.MoeLayer(4, 2, 4, 64, 32), q1, q2)):
        with pytest.raises(ValueError):
            other.forward(x, idx, alpha, a, b)
        with pytest.raises(ValueError):
            other.backward(dy, alpha, a, b)


def test_two_layers_captured_side_by_side():
    """Two layers and their optimisers, each captured into a graph of its own, replayed at once on two streams: they
    share no memory, so each repeats its own bits."""
    import pruned_expert_backward_gb300 as lrm
    T, k, E, H, I = 700, 4, 8, 256, 128
    made = []
    for n in range(2):
        x, dy, idx, alpha, w1, w2 = make(T + n, k, E, H, I)
        q1, q2 = lrm.lrm_fp8_quantize_weight(w1, glu=True), lrm.lrm_fp8_quantize_weight(w2)
        layer = lrm.MoeLayer(T + n, k, E, H, I, fp8=True)
        opt = lrm.AdamW([w1, w2], [layer.dw_gate_up, layer.dw_down], lr=0.0, weight_decay=0.0, state_bits=8,
                        max_norm=1.0, seed=n, capturable=True)

        def step(x=x, dy=dy, idx=idx, alpha=alpha, q1=q1, q2=q2, layer=layer, opt=opt):
            layer.forward(x, idx, alpha, q1, q2)
            layer.backward(dy, alpha, q1, q2)
            opt.step()

        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (layer.y, layer.dx, layer.dw_gate_up, layer.dw_down, opt.norm)]
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            step()
        made.append((graph, stream, layer, opt, want, step))
    for _ in range(5):
        for graph, stream, *_rest in made:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, layer, opt, want, _ in made:
        for got, w in zip((layer.y, layer.dx, layer.dw_gate_up, layer.dw_down, opt.norm), want):
            assert torch.equal(got, w)
        assert int(layer.dev_status.item()) == 0 and int(opt.step_dev.item()) == 6


_EVERY_CALL = r"""
import sys, torch
sys.path.insert(0, sys.argv[1]); sys.path.insert(0, sys.argv[1] + "/tests")
from pruned_expert_backward_gb300 import _lib
assert _lib.library_path().endswith(sys.argv[3])
import pruned_expert_backward_gb300 as lrm
from test_fp8_layer_gpu import make
out = []
for T, k, E, H, I in ((1, 8, 16, 512, 64), (60, 4, 8, 272, 144), (900, 2, 7, 528, 208), (4000, 2, 3, 1024, 512)):
    x, dy, idx, alpha, w1, w2 = make(T, k, E, H, I, 0.1 if T > 1 else 0.0)
    q1, q2 = lrm.lrm_fp8_quantize_weight(w1, glu=True), lrm.lrm_fp8_quantize_weight(w2)
    layer = lrm.MoeLayer(T, k, E, H, I, fp8=True)
    out.append(layer.forward(x, idx, alpha, q1, q2, residual=x).clone())
    out += layer.backward(dy, alpha, q1, q2)
    opt = lrm.AdamW([w1, w2], [layer.dw_gate_up, layer.dw_down], state_bits=8, max_norm=1.0, seed=T)
    opt.step()
    y, _ = lrm.lrm_fp8_linear(*lrm.lrm_fp8_quantize(x), q1[0][0], q1[1][0], act="swiglu", dev_status=layer.dev_status)
    out += [y, w1, w2, opt.state["m"][0].view(torch.uint8), opt.state["v_scale"][1], opt.norm]
    assert int(layer.dev_status.item()) == 0 and int(opt.dev_status.item()) == 0
torch.save([t.cpu() for t in out], sys.argv[2])
"""


def test_debug_build_checks_every_call_and_matches_release(tmp_path):
    """liblrm_debug.so runs every call with no index check failing, and gives the same bits."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    results = []
    for debug, name in (("1", "liblrm_debug.so"), ("0", "liblrm.so")):
        path = str(tmp_path / name) + ".pt"
        r = subprocess.run([sys.executable, "-c", _EVERY_CALL, root, path, "/" + name],
                           env=dict(os.environ, LRM_DEBUG=debug), capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stdout + r.stderr
        results.append(torch.load(path))
    assert len(results[0]) == len(results[1]) > 40
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_the_example_runs():
    """examples/fp8_training.py: its gradients are those of the bf16 layer but for the operands' rounding."""
    import importlib.util
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_training.py")
    spec = importlib.util.spec_from_file_location("fp8_training_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.run(tokens=600, hidden=256, inter=128, experts=16, topk=4, steps=2)
    assert r["y"] <= 0.15 and max(r["dx"], r["dw_gate_up"], r["dw_down"]) <= 0.2
    assert r["token_vs_batch"] <= 2.0 ** -7
