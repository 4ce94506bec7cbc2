"""One training step of an MoE layer, and one generated token, through the library alone.

Router product (lrm_linear with fp32 logits) -> lrm_route -> MoeLayer.forward (sort by expert, SwiGLU
product, down product, weighted way back with the block's residual) -> MoeLayer.backward, the unpruned
gradients -> PrunedBackward on the same state, which keeps the pairs with the largest LRM scores.
Prints the step's times and how far the pruned gradients are from the full ones.

    python examples/moe_layer.py [--tokens 8192] [--hidden 2048] [--inter 768] [--experts 128] [--topk 8]
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


def run(tokens=8192, hidden=2048, inter=768, experts=128, topk=8, keep=(8, 10), seed=0):
    T, H, I, E, k = tokens, hidden, inter, experts, topk
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

    x, dy = randn(T, H), randn(T, H, std=1e-3)
    w_router, b_router = randn(E, H, std=H ** -0.5), randn(E, std=0.1)
    w_gate_up, w_down = randn(E, 2 * I, H, std=H ** -0.5), randn(E, H, I, std=I ** -0.5)
    layer = lrm.MoeLayer(T, k, E, H, I)

    def forward():
        logits, _ = lrm.lrm_linear(x, w_router, bias=b_router, out_dtype=torch.float32, dev_status=layer.dev_status)
        idx, alpha, loads, quotas = lrm.lrm_route(logits, k, "ratio", *keep, dev_status=layer.dev_status)
        return idx, alpha, quotas, layer.forward(x, idx, alpha, w_gate_up, w_down, residual=x)

    idx, alpha, quotas, y = forward()
    full = [t.clone() for t in layer.backward(dy, alpha, w_gate_up, w_down)]

    # the pruned backward of the same step: it rebuilds h and phi of the kept pairs from x, and scores them
    # with the forward's norms
    _, phi_sq = lrm.lrm_swiglu_forward(layer.h_s)
    inp = {"topk_idx": idx, "alpha": alpha, "x": x, "g": dy, "w_gate_up": w_gate_up, "w_down": w_down,
           "phi_sq": phi_sq[layer.row_of_pair.long()].view(T, k)}
    pruned = lrm.PrunedBackward(T, k, E, H, I, router_grad=True, compaction="recompute")
    pruned.run(inp, quotas)
    torch.cuda.synchronize()
    for name, st in (("layer", layer.dev_status), ("pruned", pruned.dev_status)):
        if int(st.item()) != 0:
            raise RuntimeError(f"device status of the {name} path: {int(st.item())}")
    out = {"forward_ms": timed(forward), "backward_ms": timed(lambda: layer.backward(dy, alpha, w_gate_up, w_down)),
           "pruned_ms": timed(lambda: pruned.run(inp, quotas)),
           "kept": int(pruned.seg_offsets[-1]) / (T * k),
           "dx": relative(pruned.dx, full[0]), "dw_gate_up": relative(pruned.dw_gate_up, full[2]),
           "dw_down": relative(pruned.dw_down, full[3])}

    # one token at a time: the same calls without the state for a backward
    serve = lrm.MoeLayer(1, k, E, H, I, train=False)
    tok, idx1, alpha1 = x[:1].contiguous(), idx[:1].contiguous(), alpha[:1].contiguous()
    y1 = serve.forward(tok, idx1, alpha1, w_gate_up, w_down, residual=tok)
    out["token_vs_batch"] = relative(y1, y[:1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        serve.forward(tok, idx1, alpha1, w_gate_up, w_down, residual=tok)
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
    print(f"forward {r['forward_ms']:.3f} ms, backward {r['backward_ms']:.3f} ms, pruned backward "
          f"{r['pruned_ms']:.3f} ms with {r['kept']:.0%} of the pairs")
    print(f"pruned against full: dx {r['dx']:.3f}, dw_gate_up {r['dw_gate_up']:.3f}, dw_down {r['dw_down']:.3f} "
          "(relative Frobenius)")
    print(f"one token: {r['token_ms'] * 1e3:.1f} us, {r['token_vs_batch']:.1e} from its row in the batch")


if __name__ == "__main__":
    main()
