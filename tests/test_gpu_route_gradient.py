"""Gradients of the routing where a rounded score hides them, against the formulas in 64 bits, each
element in proportion to its own terms.

Tolerances, with u = 2^-23.  An exponential is within 2 u, a sum, quotient or product within u / 2;
the difference x - max that an exponential takes is rounded, |x - max| u / 2 of its value."""
import pytest
import torch

from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
NEG = float("-inf")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def confident(tokens, experts, top_k, seed):
    """Logits of which each token's top_k lie between 8 and 20, or between -20 and -8, the rest lower."""
    g = gen(seed)
    x = torch.empty(tokens, experts, device="cuda").uniform_(8, 20, generator=g)
    order = torch.rand(tokens, experts, device="cuda", generator=g).argsort(1)
    x.scatter_(1, order[:, top_k:], torch.empty(tokens, experts - top_k, device="cuda").uniform_(-60, -30, generator=g))
    x[1::2] = torch.where(x[1::2] > 0, x[1::2] - 28, x[1::2])
    return x


@pytest.mark.parametrize("experts,top_k", [(8, 1), (64, 6), (100, 12), (256, 32)])
@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_gradient_of_confident_experts(experts, top_k, renorm):
    """dx = c d s (1 - s) at logits of 8 to 20 and -20 to -8: 1 - s is as exact as s.  The bound counts two
    scores of an exponential, a sum and a quotient (3 u each) and four products: 8 u."""
    fq = require_cuda()
    x = confident(50, experts, top_k, experts + top_k)
    ids = fq.fp8q_moe_route(x, top_k, fq.SCORE_SIGMOID, renormalize=renorm)["ids"]
    d = torch.randn(50, top_k, device="cuda", generator=gen(1))
    got = fq.fp8q_moe_route_backward(x, ids, d, fq.SCORE_SIGMOID, renorm, 2.5).double().gather(1, ids.long())
    c, dd = x.double().gather(1, ids.long()), d.double()
    s, rest = 1 / (1 + torch.exp(-c)), 1 / (1 + torch.exp(c))
    if renorm:  # share_j (d_j - sum_i share_i d_i): the sums' errors count against what they add
        share = s / s.sum(1, keepdim=True)
        mean, size = (share * dd).sum(1, keepdim=True), (share * dd.abs()).sum(1, keepdim=True)
        want = 2.5 * (dd - mean) * share * rest
        tol = 2.5 * share * rest * (dd.abs() + size) * (26 + top_k) * U
    else:
        want = 2.5 * dd * s * rest
        tol = 8 * U * want.abs()
    assert ((got - want).abs() <= tol).all()
