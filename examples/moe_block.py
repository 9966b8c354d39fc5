"""A block of a network around the expert layer, on the library's operators: training and serving.

  h = x + stream,  y = norm(h)                  the stream that goes on, and what the block computes from
  weights, ids = route(y Wr^T)
  rows of the tokens, sorted by expert and quantized (both copies)
  g = rows W1[e]^T,  a = silu(gate) * up        grouped product, gated activation quantized (both copies)
  out = sum_j weights_j a W2[e]^T               grouped product, weighted sum

The backward pass ends in the gradient of x and the stream and the FP32 gradients of the weights, which are
clipped to a largest norm together.  ``decode`` takes a few tokens through the same weights: norm, route and the
whole expert layer in one call.

  python examples/moe_block.py [--tokens T] [--hidden H] [--inner I] [--experts E] [--top-k K]

prints the times of a training step and of one token.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import mxfp8_quantization_amax_gb300 as fq  # noqa: E402
from moe_layer import quantize_weights, swiglu  # noqa: E402


class MoEBlock:
    """Weights in BF16 (the norm's in FP32) with FP32 gradients; quantized copies are made once a step."""

    def __init__(self, hidden: int, inner: int, experts: int, top_k: int, device="cuda", generator=None):
        def init(*shape):
            return (torch.randn(*shape, device=device, generator=generator) * shape[-1] ** -0.5).bfloat16()

        self.experts, self.top_k = experts, top_k
        self.norm = 1.0 + 0.1 * torch.randn(hidden, device=device, generator=generator)
        self.router, self.w1, self.w2 = init(experts, hidden), init(experts, 2 * inner, hidden), init(experts, hidden, inner)
        self.begin_step()

    def begin_step(self):
        self.q1, self.q2 = quantize_weights(self.w1), quantize_weights(self.w2)

    def forward(self, x: torch.Tensor, stream: torch.Tensor):
        """x, stream [tokens, hidden] BF16: the block's output and the stream with x added."""
        n = fq.fp8q_rmsnorm(x, self.norm, stream, direction=0, want_y=True)
        y = n["y"]
        logits = (y @ self.router.t()).float()
        r = fq.fp8q_moe_route(logits, self.top_k)
        plan = fq.fp8q_moe_plan(r["ids"], self.experts, align=128)
        off, rows = plan["offsets"], plan["src"].numel()
        qy = fq.fp8q_moe_dispatch(y, plan, direction=fq.BOTH)
        # rows past the last segment are in no expert's product: they stay zero
        g = fq.fp8q_matmul_grouped(qy["q"], qy["scale_inv"], self.q1["q"], self.q1["scale_inv"], off, out=x.new_zeros(rows, self.w1.shape[1]))
        qa = fq.fp8q_swiglu(g, direction=fq.BOTH)
        e = fq.fp8q_matmul_grouped(qa["q"], qa["scale_inv"], self.q2["q"], self.q2["scale_inv"], off, out=x.new_zeros(rows, x.shape[1]))
        self.kept = (n, logits, r, plan, qy, g, qa, e)
        return fq.fp8q_moe_combine(e, plan, r["weights"]), n["h"]

    def backward(self, d_out: torch.Tensor, d_stream: torch.Tensor, max_norm: float | None = None) -> dict:
        """The gradients of x (BF16, the stream's too) and of the weights (FP32, clipped together to max_norm)."""
        n, logits, r, plan, qy, g, qa, e = self.kept
        off, zeros = plan["offsets"], d_out.new_zeros
        c = fq.fp8q_moe_combine_backward(d_out, e, plan, r["weights"])
        qe = fq.fp8q_quantize_blockwise(c["d_y"], fq.E5M2, direction=fq.BOTH)
        d_a = fq.fp8q_matmul_grouped(qe["q"], qe["scale_inv"], self.q2["q_t"], self.q2["scale_inv_t"], off, a_fmt=fq.E5M2,
                                     out=zeros(g.shape[0], self.w2.shape[2]))
        d_w2 = fq.fp8q_matmul_grouped_wgrad(qe["q_t"], qe["scale_inv_t"], qa["q_t"], qa["scale_inv_t"], off, a_fmt=fq.E5M2)
        qg = fq.fp8q_swiglu_backward(g, d_a, fmt=fq.E5M2, direction=fq.BOTH)
        d_rows = fq.fp8q_matmul_grouped(qg["q"], qg["scale_inv"], self.q1["q_t"], self.q1["scale_inv_t"], off, a_fmt=fq.E5M2,
                                        out=zeros(g.shape[0], d_out.shape[1]))
        d_w1 = fq.fp8q_matmul_grouped_wgrad(qg["q_t"], qg["scale_inv_t"], qy["q_t"], qy["scale_inv_t"], off, a_fmt=fq.E5M2)
        d_logits = fq.fp8q_moe_route_backward(logits, r["ids"], c["d_weights"]).bfloat16()
        d_y = (fq.fp8q_moe_combine(d_rows, plan).float() + (d_logits @ self.router).float()).bfloat16()
        d = fq.fp8q_rmsnorm_backward(d_y, n["h"], self.norm, n["rstd"], d_h=d_stream)
        grads = {"norm": d["d_weight"], "router": (d_logits.t() @ n["y"]).float(), "w1": d_w1, "w2": d_w2}
        if max_norm is not None:
            weights = list(grads.values())
            fq.fp8q_clip_grads(weights, max_norm, out=weights)
        return {"x": d["d_x"], **grads}

    def decode(self, x: torch.Tensor, stream: torch.Tensor):
        """forward() for up to 64 tokens while serving."""
        n = fq.fp8q_rmsnorm(x, self.norm, stream, direction=0, want_y=True)
        r = fq.fp8q_moe_route((n["y"] @ self.router.t()).float(), self.top_k)
        out = fq.fp8q_moe_decode(n["y"], r["ids"], r["weights"], self.q1["q"], self.q1["scale_inv"], self.q2["q"], self.q2["scale_inv"])
        return out, n["h"]


def reference(block: MoEBlock, x, stream, d_out, d_stream, ids) -> dict:
    """The same block in FP32, with the given choice of experts: out, the stream and the gradients."""
    ids = ids.long()
    h = (x.float() + stream.float()).bfloat16().float().requires_grad_(True)
    norm, router, w1, w2 = (t.float().detach().requires_grad_(True) for t in (block.norm, block.router, block.w1, block.w2))
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * norm
    w = torch.softmax((y @ router.t()).gather(1, ids), 1)  # renormalised softmax weights
    out = torch.zeros_like(y)
    for e in range(block.experts):
        t, j = (ids == e).nonzero(as_tuple=True)
        out = out.index_add(0, t, w[t, j, None] * (swiglu(y[t] @ w1[e].t()) @ w2[e].t()))
    g = torch.autograd.grad((out, h), (h, norm, router, w1, w2), (d_out.float(), d_stream.float()))
    return dict(zip(("out", "stream", "x", "norm", "router", "w1", "w2"), (out.detach(), h.detach(), *g)))


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("tokens", 4096), ("hidden", 2048), ("inner", 1024), ("experts", 16), ("top-k", 4), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(0)
    block = MoEBlock(a.hidden, a.inner, a.experts, a.top_k, generator=gen)
    x, stream = (torch.randn(a.tokens, a.hidden, device="cuda", generator=gen).bfloat16() for _ in range(2))
    d_out, d_stream = ((torch.randn(a.tokens, a.hidden, device="cuda", generator=gen) / a.tokens).bfloat16() for _ in range(2))
    out, h = block.forward(x, stream)
    got = {"out": out, "stream": h, **block.backward(d_out, d_stream)}
    for name, v in reference(block, x, stream, d_out, d_stream, block.kept[2]["ids"]).items():
        print("%-7s off by %.3f (norm of the difference over the norm)" % (name, ((got[name].float() - v).norm() / v.norm()).item()))
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for label, steps, run in (("a training step", a.steps, lambda: (block.begin_step(), block.forward(x, stream), block.backward(d_out, d_stream, 1.0))),
                              ("one token", 20 * a.steps, lambda: block.decode(x[:1], stream[:1]))):
        for i in range(steps + 3):
            if i == 3:
                start.record()
            run()
        end.record()
        fq.check_device()
        print("%s takes %.3f ms" % (label, start.elapsed_time(end) / steps))


if __name__ == "__main__":
    main()
