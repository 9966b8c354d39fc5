"""The block of examples/moe_block.py, training and serving, against the block in FP32.

Bounds, on the norm of the difference over the norm, as for the expert layer alone: a product of values
rounded to E4M3 is off by at most E4 = sqrt(2^-8 + 2^-8) (half a unit of 3 mantissa bits in each factor), one
with an E5M2 factor by E5 = sqrt(2^-6 + 2^-8), errors of a chain add in the norm at worst and a BF16 rounding
adds 2^-8: the norm's output has one.  The few-token layer rounds the weights alone, 2^-4 a product."""
import os
import sys

import pytest
import torch

from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

E4 = (2 ** -8 + 2 ** -8) ** 0.5   # one product, both factors E4M3
E5 = (2 ** -6 + 2 ** -8) ** 0.5   # one factor E5M2


def make(tokens, hidden, inner, experts, top_k):
    import moe_block

    g = torch.Generator(device="cuda").manual_seed(tokens)
    block = moe_block.MoEBlock(hidden, inner, experts, top_k, generator=g)
    return moe_block, block, [torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16() for _ in range(4)]


def off(got, want):
    return ((got.float() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("tokens,hidden,inner,experts,top_k", [(64, 256, 128, 4, 2), (301, 272, 144, 7, 3), (16, 512, 256, 40, 8)])
def test_training_against_fp32(tokens, hidden, inner, experts, top_k):
    require_cuda()
    moe_block, block, (x, stream, d_out, d_stream) = make(tokens, hidden, inner, experts, top_k)
    out, h = block.forward(x, stream)
    got = {"out": out, "stream": h, **block.backward(d_out, d_stream)}
    want = moe_block.reference(block, x, stream, d_out, d_stream, block.kept[2]["ids"])
    assert torch.equal(got["stream"].float(), want.pop("stream"))
    hh = E4 + 2 * 2 ** -8             # of the first product; of the activation twice that, and a rounding
    o = 2 * hh + 2 ** -8 + E4 + 2 ** -7
    d_a = E5 + 2 ** -7
    d_h = d_a + 2 * hh + 2 ** -7      # times the derivatives of silu and the other branch
    d_y = 1.5 * (E5 + d_h + 2 ** -7)  # of the experts' and the routing's part
    # the norm's own gradients pass it on, rows and columns weighted by factors within 1.3 of each other; d_stream, exact, adds to the norm below
    bound = {"out": o, "w2": E5 + 2 * hh + 2 ** -7, "w1": E5 + d_h + 2 ** -7, "x": 1.3 * d_y + 2 ** -7, "norm": 1.3 * d_y + 2 ** -7, "router": 4 * o}
    for name, v in want.items():
        assert off(got[name], v) < bound[name], (name, off(got[name], v), bound[name])


def test_clipped_together():
    """The weights' gradients are scaled by one factor, to the largest norm."""
    require_cuda()
    _, block, (x, stream, d_out, d_stream) = make(64, 256, 128, 4, 2)
    block.forward(x, stream)
    plain, clipped = block.backward(d_out, d_stream), block.backward(d_out, d_stream, 0.25)
    names = ("norm", "router", "w1", "w2")
    norm = sum(float(plain[k].double().square().sum()) for k in names) ** 0.5
    assert norm > 0.25
    for k in names:
        assert torch.allclose(clipped[k], plain[k] * (0.25 / (norm + 1e-6)), rtol=2 ** -17, atol=0)
    assert torch.equal(clipped["x"], plain["x"])


@pytest.mark.parametrize("tokens,hidden,inner,experts,top_k", [(1, 256, 128, 4, 2), (7, 272, 144, 7, 3), (64, 512, 256, 40, 8)])
def test_serving_against_fp32_and_training(tokens, hidden, inner, experts, top_k):
    require_cuda()
    moe_block, block, (x, stream, d_out, d_stream) = make(tokens, hidden, inner, experts, top_k)
    out, h = block.decode(x, stream)
    trained, h2 = block.forward(x, stream)
    assert torch.equal(h, h2)
    want = moe_block.reference(block, x, stream, d_out, d_stream, block.kept[2]["ids"])["out"]
    assert off(out, want) < 3 * 2 ** -4 + 2 ** -6
    assert off(trained, want) < 3 * E4 + 2 ** -5


def test_serving_in_a_graph():
    require_cuda()
    _, block, (x, stream, *_) = make(4, 256, 128, 8, 2)
    block.decode(x, stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, h = block.decode(x, stream)
    for seed in range(2):
        x.copy_(torch.randn(4, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)))
        graph.replay()
        now = block.decode(x, stream)
        assert torch.equal(out, now[0]) and torch.equal(h, now[1])
