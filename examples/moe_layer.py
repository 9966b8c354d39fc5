"""One expert layer in blockwise FP8, forward and backward, on the library's operators.

  logits = x Wr^T                               (torch: a small BF16 product)
  weights, ids = route(logits)                  softmax, top-k, renormalised
  rows of the tokens, sorted by expert and quantized in one pass (both copies)
  h = rows W1[e]^T,  a = silu(gate) * up        grouped product, elementwise in torch
  y = a W2[e]^T                                 grouped product
  out = sum_j weights_j y_j                     combine

The backward pass uses the transposed copies: Dgrad with the weights' 128x128
blocks transposed, Wgrad over each expert's rows (segments padded to 128), the
weighted sum's gradients, and the routing's.

  python examples/moe_layer.py [--tokens T] [--hidden H] [--inner I] [--experts E] [--top-k K]

prints the time of a step and how far it is from the layer in FP32.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp8_quantization_amax_gb300 as fq  # noqa: E402


def quantize_weights(w: torch.Tensor) -> dict:
    """w [experts, n, k] BF16 in 128x128 blocks: q [experts, n, k], q_t [experts, k, n] and their scales."""
    e, n, k = w.shape
    bn, bk = -(-n // 128), -(-k // 128)
    out = {"q": torch.empty(e, n, k, dtype=torch.uint8, device=w.device), "scale_inv": torch.empty(e, bn, bk, device=w.device),
           "q_t": torch.empty(e, k, n, dtype=torch.uint8, device=w.device), "scale_inv_t": torch.empty(e, bk, bn, device=w.device)}
    for i in range(e):
        fq.fp8q_quantize_blockwise(w[i], block=fq.BLOCK_128X128, direction=fq.BOTH, out={name: t[i] for name, t in out.items()})
    return out


def swiglu(h: torch.Tensor) -> torch.Tensor:
    gate, up = h.chunk(2, 1)
    return torch.nn.functional.silu(gate) * up


class MoELayer:
    """Weights in BF16 with FP32 gradients; quantized copies are made once a step (``begin_step``)."""

    def __init__(self, hidden: int, inner: int, experts: int, top_k: int, device="cuda", generator=None):
        def init(*shape):
            return (torch.randn(*shape, device=device, generator=generator) * shape[-1] ** -0.5).bfloat16()

        self.experts, self.top_k = experts, top_k
        self.router, self.w1, self.w2 = init(experts, hidden), init(experts, 2 * inner, hidden), init(experts, hidden, inner)
        self.begin_step()

    def begin_step(self):
        self.q1, self.q2 = quantize_weights(self.w1), quantize_weights(self.w2)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x [tokens, hidden] BF16; keeps what the backward pass needs."""
        logits = (x @ self.router.t()).float()
        r = fq.fp8q_moe_route(logits, self.top_k)
        plan = fq.fp8q_moe_plan(r["ids"], self.experts, align=128)
        off = plan["offsets"]
        qx = fq.fp8q_moe_dispatch(x, plan, direction=fq.BOTH)
        rows = plan["src"].numel()
        # rows past the last segment are in no expert's product: they stay zero
        h = fq.fp8q_matmul_grouped(qx["q"], qx["scale_inv"], self.q1["q"], self.q1["scale_inv"], off,
                                   out=x.new_zeros(rows, self.w1.shape[1]))
        a = swiglu(h)
        qa = fq.fp8q_quantize_blockwise(a, direction=fq.BOTH)
        y = fq.fp8q_matmul_grouped(qa["q"], qa["scale_inv"], self.q2["q"], self.q2["scale_inv"], off,
                                   out=x.new_zeros(rows, x.shape[1]))
        out = fq.fp8q_moe_combine(y, plan, r["weights"])
        self.kept = (x, logits, r, plan, qx, h, qa, y)
        return out

    def backward(self, d_out: torch.Tensor) -> dict:
        """The gradients of x (BF16) and of the weights (FP32)."""
        x, logits, r, plan, qx, h, qa, y = self.kept
        off = plan["offsets"]
        g = fq.fp8q_moe_combine_backward(d_out, y, plan, r["weights"])
        qy = fq.fp8q_quantize_blockwise(g["d_y"], fq.E5M2, direction=fq.BOTH)
        d_a = fq.fp8q_matmul_grouped(qy["q"], qy["scale_inv"], self.q2["q_t"], self.q2["scale_inv_t"], off, a_fmt=fq.E5M2,
                                     out=x.new_zeros(h.shape[0], self.w2.shape[2]))
        d_w2 = fq.fp8q_matmul_grouped_wgrad(qy["q_t"], qy["scale_inv_t"], qa["q_t"], qa["scale_inv_t"], off, a_fmt=fq.E5M2)
        leaf = h.detach().requires_grad_(True)
        (d_h,) = torch.autograd.grad(swiglu(leaf), leaf, d_a)
        qh = fq.fp8q_quantize_blockwise(d_h, fq.E5M2, direction=fq.BOTH)
        d_rows = fq.fp8q_matmul_grouped(qh["q"], qh["scale_inv"], self.q1["q_t"], self.q1["scale_inv_t"], off, a_fmt=fq.E5M2,
                                        out=x.new_zeros(h.shape[0], x.shape[1]))
        d_w1 = fq.fp8q_matmul_grouped_wgrad(qh["q_t"], qh["scale_inv_t"], qx["q_t"], qx["scale_inv_t"], off, a_fmt=fq.E5M2)
        d_logits = fq.fp8q_moe_route_backward(logits, r["ids"], g["d_weights"]).bfloat16()
        d_x = fq.fp8q_moe_combine(d_rows, plan).float() + (d_logits @ self.router).float()
        return {"x": d_x.bfloat16(), "router": (d_logits.t() @ x).float(), "w1": d_w1, "w2": d_w2}


def reference(layer: MoELayer, x: torch.Tensor, d_out: torch.Tensor) -> dict:
    """The same layer in FP32, with the layer's choice of experts: out and the gradients."""
    ids = layer.kept[2]["ids"].long()
    x, router, w1, w2 = (t.float().requires_grad_(True) for t in (x, layer.router, layer.w1, layer.w2))
    w = torch.softmax((x @ router.t()).gather(1, ids), 1)  # renormalised softmax weights
    out = torch.zeros_like(x)
    for e in range(layer.experts):
        t, j = (ids == e).nonzero(as_tuple=True)
        out = out.index_add(0, t, w[t, j, None] * (swiglu(x[t] @ w1[e].t()) @ w2[e].t()))
    g = torch.autograd.grad(out, (x, router, w1, w2), d_out.float())
    return dict(zip(("out", "x", "router", "w1", "w2"), (out.detach(), *g)))


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("tokens", 4096), ("hidden", 2048), ("inner", 1024), ("experts", 16), ("top-k", 4), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    layer = MoELayer(a.hidden, a.inner, a.experts, a.top_k, generator=g)
    x = torch.randn(a.tokens, a.hidden, device="cuda", generator=g).bfloat16()
    d_out = (torch.randn(a.tokens, a.hidden, device="cuda", generator=g) / a.tokens).bfloat16()
    got = {"out": layer.forward(x), **layer.backward(d_out)}
    want = reference(layer, x, d_out)
    for name, v in want.items():
        print("%-7s off by %.3f (norm of the difference over the norm)" % (name, ((got[name].float() - v).norm() / v.norm()).item()))
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for i in range(a.steps + 3):
        if i == 3:
            start.record()
        layer.begin_step()
        layer.forward(x)
        layer.backward(d_out)
    end.record()
    fq.check_device()
    print("a step takes %.2f ms" % (start.elapsed_time(end) / a.steps))


if __name__ == "__main__":
    main()
