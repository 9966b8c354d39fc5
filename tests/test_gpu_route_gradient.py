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


@pytest.mark.parametrize("experts,top_k", [(5, 2), (64, 8), (100, 12), (257, 3), (1000, 32)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_is_nan_where_the_weights_are(experts, top_k, score, renorm, dtype):
    """A token whose weights routing made NaN gets NaN for every logit; its neighbours keep their gradients bit
    for bit, whether a row starts on 16 bytes or not."""
    fq = require_cuda()
    x = torch.randn(23, experts, device="cuda", generator=gen(experts)).to(dtype)
    d = torch.randn(23, top_k, device="cuda", generator=gen(2))
    clean = fq.fp8q_moe_route(x, top_k, score, renormalize=renorm)
    want = fq.fp8q_moe_route_backward(x, clean["ids"], d, score, renorm)
    bad = x.clone()
    lowest = x.float().argmin(1)  # chosen by nobody (of 5 experts 2 are chosen)
    bad[2, lowest[2]] = float("nan")
    bad[3, clean["ids"][3, 0].long()] = float("nan")
    bad[9] = NEG
    bad[9, experts - 1] = float("nan")  # a NaN is all there is
    bad[16, 0] = -float("nan")
    bad[22, experts // 2] = float("inf")
    r = fq.fp8q_moe_route(bad, top_k, score, renormalize=renorm)
    got = fq.fp8q_moe_route_backward(bad, r["ids"], d, score, renorm)
    poisoned = torch.isnan(r["weights"]).any(1)
    assert poisoned.nonzero()[:, 0].tolist() == [2, 3, 9, 16] + ([22] if score == 0 else [])
    assert torch.isnan(got[poisoned]).all()
    assert torch.isfinite(got[~poisoned]).all()
    same = [t for t in range(23) if t not in (2, 3, 9, 16, 22)]
    assert torch.equal(got[same], want[same])
    # a buffer that starts off a 16-byte boundary
    raw = torch.empty(23 * experts + 1, dtype=dtype, device="cuda")
    off = fq.fp8q_moe_route_backward(bad, r["ids"], d, score, renorm, out=raw[1:].view(23, experts))
    assert torch.equal(torch.nan_to_num(off.float(), nan=7e7), torch.nan_to_num(got.float(), nan=7e7))
