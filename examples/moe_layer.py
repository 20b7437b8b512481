"""A mixture-of-experts layer on block-scaled FP8 weights, as a serving program would run it.

    python examples/moe_layer.py [--tokens 256] [--hidden 2048] [--width 1408] [--experts 64] [--chosen 8]

Once, at load: the router's and the experts' bf16 weights are quantized with a scale for each 128 x 128
block. Every step: the router's logits (a block-scaled linear), the choice of experts, the chosen
experts' networks and their weighted sum. Random weights; prints the time of a step and how far the
layer is from the same layer in fp32 on the unquantized weights.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_w8a8_quantized_dynamic_gb300 as F  # noqa: E402


class MoELayer:
    """gate bf16 [E, H], w13 bf16 [E, 2, I, H] (gate and up), w2 bf16 [E, H, I]."""

    def __init__(self, gate, w13, w2, chosen: int, bias=None):
        self.chosen, self.bias = chosen, bias
        self.gate = F.fp8_block_quantize_weight(gate)
        self.w13 = F.fp8_block_quantize_weight(w13)
        self.w2 = F.fp8_block_quantize_weight(w2)
        self.shape = (gate.shape[0], gate.shape[1], w13.shape[2])  # E, H, I

    def workspace(self, tokens: int, device):
        """Scratch for steps of up to `tokens` tokens, kept by the caller."""
        E, H, I = self.shape
        need = max(max(F.fp8_block_workspace_bytes(t, H, E), F.fp8_moe_workspace_bytes(t, self.chosen, E, H, I))
                   for t in range(1, tokens + 1))
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)

    def __call__(self, x, ws=None):
        logits = F.fp8_block_linear(x, *self.gate, ws=ws)
        ids, weights = F.fp8_moe_route(logits, self.chosen, score="sigmoid", bias=self.bias, renormalize=True)
        return F.fp8_moe_experts(x, ids, weights, *self.w13, *self.w2, ws=ws), ids, weights


def random_weights(E: int, H: int, I: int, seed: int, device):
    g = torch.Generator(device=device).manual_seed(seed)

    def draw(*shape, std):
        return (torch.randn(shape, generator=g, device=device) * std).to(torch.bfloat16)

    return draw(E, H, std=H ** -0.5), draw(E, 2, I, H, std=H ** -0.5), draw(E, H, I, std=I ** -0.5)


def in_fp32(x, gate, w13, w2, ids, weights):
    """The layer on the bf16 weights, fp32 throughout, for the experts that `ids` names."""
    x = x.float()
    y = torch.zeros_like(x)
    for e in range(w13.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            g, u = x[t] @ w13[e, 0].float().T, x[t] @ w13[e, 1].float().T
            y.index_add_(0, t, (torch.nn.functional.silu(g) * u) @ w2[e].float().T * weights[t, j][:, None])
    return y


def main(argv=None) -> float:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 256), ("hidden", 2048), ("width", 1408), ("experts", 64), ("chosen", 8), ("steps", 50)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    device = "cuda:0"
    weights = random_weights(a.experts, a.hidden, a.width, 1, device)
    layer = MoELayer(*weights, a.chosen, bias=torch.zeros(a.experts, device=device))
    x = torch.randn(a.tokens, a.hidden, device=device).to(torch.bfloat16)
    ws = layer.workspace(a.tokens, device)
    y, ids, w = layer(x, ws)
    ref = in_fp32(x, *weights, ids, w)
    off = float((y.float() - ref).norm() / ref.norm())
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(3):
        layer(x, ws)
    torch.cuda.synchronize()
    start.record()
    for _ in range(a.steps):
        layer(x, ws)
    stop.record()
    torch.cuda.synchronize()
    assert F.fp8_last_device_status() == F.FP8_OK
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.width}, {a.chosen} chosen: "
          f"{start.elapsed_time(stop) / a.steps * 1e3:.1f} us a step, relative difference to fp32 {off:.3f}")
    return off


if __name__ == "__main__":
    main()
