"""The expert layer of examples/moe_layer.py, forward and backward, against 64 bits.

The quantizers' copies are taken as the layer made them, so that what is left is the operators' own
arithmetic and BF16 roundings of 2^-9: a missing or misplaced term is two orders of magnitude larger than any
bound here."""
import os
import sys

import pytest
import torch

from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

FP8 = (torch.float8_e4m3fn, torch.float8_e5m2)
R = 2.0 ** -9  # half a unit of BF16, as a share of a value


def decoded(q, scale, fmt, block):
    r = torch.arange(q.shape[-2], device="cuda") // block
    c = torch.arange(q.shape[-1], device="cuda") // 128
    return q.view(FP8[fmt]).double() * scale.double()[..., r, :][..., c]


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("tokens,hidden,inner,experts,top_k", [(64, 256, 128, 4, 2), (301, 272, 144, 7, 3), (16, 512, 256, 40, 8), (700, 384, 272, 3, 2)])
def test_every_step_of_the_layer(monkeypatch, tokens, hidden, inner, experts, top_k):
    fq = require_cuda()
    import moe_layer

    g = torch.Generator(device="cuda").manual_seed(tokens)
    layer = moe_layer.MoELayer(hidden, inner, experts, top_k, generator=g)
    x = torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16()
    d_out = torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16()
    copies, rows_grad = [], []
    quantize, combine = fq.fp8q_quantize_blockwise, fq.fp8q_moe_combine
    monkeypatch.setattr(fq, "fp8q_quantize_blockwise", lambda *a, **k: copies.append(quantize(*a, **k)) or copies[-1])
    monkeypatch.setattr(fq, "fp8q_moe_combine", lambda y, *a, **k: rows_grad.append(y) or combine(y, *a, **k))
    got = {"out": layer.forward(x), **layer.backward(d_out)}
    fq.check_device()
    qa, qy, qh = copies
    _, logits, r, plan, qx, h, _, y = layer.kept
    ids, at, offsets = r["ids"].long(), plan["row_of"].long(), plan["offsets"].tolist()
    src = plan["src"].long()
    real = src >= 0
    of_row = torch.zeros(src.numel(), dtype=torch.long, device="cuda")
    for e in range(experts):
        of_row[offsets[e]:offsets[e + 1]] = e
    assert torch.equal(of_row[at], ids) and torch.equal(src[at.reshape(-1)], torch.arange(ids.numel(), device="cuda"))

    # forward
    xs, xt = decoded(qx["q"], qx["scale_inv"], 0, 1), decoded(qx["q_t"], qx["scale_inv_t"], 0, 1).T
    w1, w2 = decoded(layer.q1["q"], layer.q1["scale_inv"], 0, 128), decoded(layer.q2["q"], layer.q2["scale_inv"], 0, 128)
    # a row of codes is within half a unit of 3 mantissa bits, and so is its transposed copy
    assert off(xs[at], x.double()[:, None].expand(-1, top_k, -1)) < 2 ** -4 and off(xt[at], x.double()[:, None].expand(-1, top_k, -1)) < 2 ** -4
    assert (xs[~real] == 0).all() and (xt[~real] == 0).all()
    assert off(w1, layer.w1.double()) < 2 ** -4 and off(w2, layer.w2.double()) < 2 ** -4
    weights = torch.softmax(logits.double().gather(1, ids), 1)
    assert off(logits, x.double() @ layer.router.double().T) < 2 * R
    assert off(r["weights"], weights) < 1e-5

    def per_row(rows, mats):
        out = torch.zeros(rows.shape[0], mats.shape[1], dtype=torch.float64, device="cuda")
        for e in range(experts):
            out[offsets[e]:offsets[e + 1]] = rows[offsets[e]:offsets[e + 1]] @ mats[e].T
        return out

    h64 = per_row(xs, w1)
    assert off(h, h64) < 2 * R
    a64 = torch.nn.functional.silu(h.double()[:, :inner]) * h.double()[:, inner:]
    a, a_t = decoded(qa["q"], qa["scale_inv"], 0, 1), decoded(qa["q_t"], qa["scale_inv_t"], 0, 1).T
    assert off(a, a64) < 2 ** -4 + 4 * R and off(a_t, a64) < 2 ** -4 + 4 * R
    y64 = per_row(a, w2)
    assert off(y, y64) < 2 * R
    assert off(got["out"], (y64[at] * weights[:, :, None]).sum(1)) < 4 * R

    # backward
    d64 = d_out.double()
    d_w64 = (y.double()[at] * d64[:, None, :]).sum(2)
    d_y64 = torch.zeros_like(y64)
    d_y64[at.reshape(-1)] = (weights[:, :, None] * d64[:, None, :]).reshape(-1, hidden)
    d_y, d_y_t = decoded(qy["q"], qy["scale_inv"], 1, 1), decoded(qy["q_t"], qy["scale_inv_t"], 1, 1).T
    assert off(d_y, d_y64) < 2 ** -3 + 2 * R and off(d_y_t, d_y64) < 2 ** -3 + 2 * R
    assert (d_y[~real] == 0).all() and (d_y_t[~real] == 0).all()
    w1_t, w2_t = decoded(layer.q1["q_t"], layer.q1["scale_inv_t"], 0, 128), decoded(layer.q2["q_t"], layer.q2["scale_inv_t"], 0, 128)
    assert torch.equal(w1_t, w1.transpose(1, 2)) and torch.equal(w2_t, w2.transpose(1, 2))
    d_a64 = per_row(d_y, w2_t)
    leaf = h.double().requires_grad_(True)
    (d_h64,) = torch.autograd.grad(torch.nn.functional.silu(leaf[:, :inner]) * leaf[:, inner:], leaf, d_a64)
    d_h, d_h_t = decoded(qh["q"], qh["scale_inv"], 1, 1), decoded(qh["q_t"], qh["scale_inv_t"], 1, 1).T
    # d_a, silu's derivative and d_h are rounded to BF16 on the way
    assert off(d_h, d_h64) < 2 ** -3 + 8 * R and off(d_h_t, d_h64) < 2 ** -3 + 8 * R
    for name, left, right in (("w2", d_y_t, a_t), ("w1", d_h_t, xt)):
        want = torch.stack([left[offsets[e]:offsets[e + 1]].T @ right[offsets[e]:offsets[e + 1]] for e in range(experts)])
        assert off(got[name], want) < 1e-5, name
    d_rows64 = per_row(d_h, w1_t)
    assert len(rows_grad) == 2 and off(rows_grad[1][real], d_rows64[real]) < 2 * R
    # the routing's gradient: one rounding of d_logits and one of the product, in each of which errors of independent
    # signs grow no further; its share of d_x is compared with nothing else in the way
    mean = (weights * d_w64).sum(1, keepdim=True)
    d_logits = torch.zeros_like(logits, dtype=torch.float64).scatter(1, ids, weights * (d_w64 - mean))
    assert off(got["router"], d_logits.T @ x.double()) < 4 * R
    term = d_logits @ layer.router.double()
    rows_part = d_rows64[at].sum(1)
    want = rows_part + term
    assert off(got["x"], want) < 4 * R
    left = (got["x"].double() - combine(rows_grad[1], plan).double())
    bound = 4 * R * (want.norm() + 2 * rows_part.norm()) / term.norm()  # roundings of d_x and of its two parts
    assert off(left, term) < bound < 0.5
