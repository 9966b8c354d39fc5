"""The expert layer of examples/moe_layer.py against the layer in FP32.

Bounds, on the norm of the difference over the norm: a product of values rounded to E4M3 is off by
at most sqrt(2^-8 + 2^-8) (half a unit of 3 mantissa bits in each factor), one with an E5M2 factor
by sqrt(2^-6 + 2^-8).  Errors of a chain add in the norm at worst; a BF16 rounding adds 2^-8; the
elementwise product of the gate and the up branch counts its two errors."""
import os
import sys

import pytest
import torch

from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

E4 = (2 ** -8 + 2 ** -8) ** 0.5   # one product, both factors E4M3
E5 = (2 ** -6 + 2 ** -8) ** 0.5   # one factor E5M2


@pytest.mark.parametrize("tokens,hidden,inner,experts,top_k", [(64, 256, 128, 4, 2), (301, 272, 144, 7, 3), (16, 512, 256, 40, 8)])
def test_layer_against_fp32(tokens, hidden, inner, experts, top_k):
    require_cuda()
    import moe_layer

    g = torch.Generator(device="cuda").manual_seed(tokens)
    layer = moe_layer.MoELayer(hidden, inner, experts, top_k, generator=g)
    x = torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16()
    d_out = torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16()
    got = {"out": layer.forward(x), **layer.backward(d_out)}
    want = moe_layer.reference(layer, x, d_out)
    h = E4 + 2 ** -8                  # of h; of a = silu(gate) * up twice that, and a rounding
    out = 2 * h + 2 ** -8 + E4 + 2 ** -7
    d_a = E5 + 2 ** -7
    d_h = d_a + 2 * h + 2 ** -7       # times the derivatives of silu and the other branch
    bound = {"out": out, "w2": E5 + 2 * h + 2 ** -7, "w1": E5 + d_h + 2 ** -8, "x": 1.5 * (E5 + d_h + 2 ** -7), "router": 4 * out}
    for name, v in want.items():
        off = ((got[name].float() - v).norm() / v.norm()).item()
        assert off < bound[name], (name, off, bound[name])
