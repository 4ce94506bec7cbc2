"""Training steps of an MoE layer in 8 bits, and one generated token, through the library alone.

Router product and routing -> MoeLayer(fp8=True): rows and weights in e4m3 with a scale for each block of 128, the
products and their rows' gradients on the 8-bit tensor cores, the weights' gradients from the bf16 rows -> AdamW over
the router's and the experts' weights in one call, clipped by their common norm, with 8-bit states ->
lrm_fp8_quantize_weight for the next step.  Prints the step's times beside the bf16 layer's and how far the first
step's outputs and gradients are from it.

    python examples/fp8_training.py [--tokens 8192] [--hidden 2048] [--inter 768] [--experts 128] [--topk 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import pruned_expert_backward_gb300 as lrm  # noqa: E402


def timed(f, n=5):
    f()
    a, b = torch.cuda.Event(True), torch.cuda.Event(True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def relative(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def run(tokens=8192, hidden=2048, inter=768, experts=128, topk=8, steps=3, seed=0):
    T, H, I, E, k = tokens, hidden, inter, experts, topk
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

    x, dy = randn(T, H), randn(T, H, std=1e-3)
    w_router = randn(E, H, std=H ** -0.5)
    w_gate_up, w_down = randn(E, 2 * I, H, std=H ** -0.5), randn(E, H, I, std=I ** -0.5)
    q_gate_up, q_down = lrm.lrm_fp8_quantize_weight(w_gate_up, glu=True), lrm.lrm_fp8_quantize_weight(w_down)
    layer, full = lrm.MoeLayer(T, k, E, H, I, fp8=True), lrm.MoeLayer(T, k, E, H, I)
    optimiser = lrm.AdamW([w_gate_up, w_down], [layer.dw_gate_up, layer.dw_down], lr=1e-4, betas=(0.9, 0.95),
                          weight_decay=0.1, state_bits=8, max_norm=1.0, seed=seed)

    def route():
        logits, _ = lrm.lrm_linear(x, w_router, out_dtype=torch.float32, dev_status=layer.dev_status)
        return lrm.lrm_route(logits, k, "ratio", 1, 1, dev_status=layer.dev_status)[:2]

    idx, alpha = route()

    def forward():
        return layer.forward(x, idx, alpha, q_gate_up, q_down, residual=x)

    def update():
        optimiser.step()
        lrm.lrm_fp8_quantize_weight(w_gate_up, glu=True, q=q_gate_up[0], scale=q_gate_up[1])
        lrm.lrm_fp8_quantize_weight(w_down, q=q_down[0], scale=q_down[1])

    # the first step beside the bf16 layer's
    y = forward()
    dx, _, dw_gate_up, dw_down = layer.backward(dy, alpha, q_gate_up, q_down)
    y_full = full.forward(x, idx, alpha, w_gate_up, w_down, residual=x)
    dx_full, _, dw_gate_up_full, dw_down_full = full.backward(dy, alpha, w_gate_up, w_down)
    out = {"y": relative(y - x, y_full - x), "dx": relative(dx, dx_full),
           "dw_gate_up": relative(dw_gate_up, dw_gate_up_full), "dw_down": relative(dw_down, dw_down_full)}
    out["forward_ms"], out["full_forward_ms"] = timed(forward), timed(
        lambda: full.forward(x, idx, alpha, w_gate_up, w_down, residual=x))
    out["backward_ms"] = timed(lambda: layer.backward(dy, alpha, q_gate_up, q_down))
    out["full_backward_ms"] = timed(lambda: full.backward(dy, alpha, w_gate_up, w_down))
    for _ in range(steps):
        forward()
        layer.backward(dy, alpha, q_gate_up, q_down)
        update()
    out["update_ms"] = timed(update)
    torch.cuda.synchronize()
    for name, st in (("layer", layer.dev_status), ("optimiser", optimiser.dev_status)):
        if int(st.item()) != 0:
            raise RuntimeError(f"device status of the {name}: {int(st.item())}")

    # one token at a time
    y = forward()
    serve = lrm.MoeLayer(1, k, E, H, I, train=False, fp8=True)
    tok, idx1, alpha1 = x[:1].contiguous(), idx[:1].contiguous(), alpha[:1].contiguous()
    out["token_vs_batch"] = relative(serve.forward(tok, idx1, alpha1, q_gate_up, q_down, residual=tok), y[:1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        serve.forward(tok, idx1, alpha1, q_gate_up, q_down, residual=tok)
    out["token_ms"] = timed(graph.replay, 20)
    return out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=8192)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=768)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--topk", type=int, default=8)
    a = ap.parse_args()
    r = run(a.tokens, a.hidden, a.inter, a.experts, a.topk)
    print(f"forward {r['forward_ms']:.3f} ms (bf16 {r['full_forward_ms']:.3f}), backward {r['backward_ms']:.3f} ms "
          f"(bf16 {r['full_backward_ms']:.3f}), update {r['update_ms']:.3f} ms")
    print(f"8 bits against bf16: y {r['y']:.3f}, dx {r['dx']:.3f}, dw_gate_up {r['dw_gate_up']:.3f}, "
          f"dw_down {r['dw_down']:.3f} (relative Frobenius)")
    print(f"one token: {r['token_ms'] * 1e3:.1f} us, {r['token_vs_batch']:.1e} from its row in the batch")


if __name__ == "__main__":
    main()
