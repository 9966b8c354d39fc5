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


def dominant(tokens, experts, seed):
    """Logits of which one a token lies 4 to 24 above the best of the others, which span 8."""
    g = gen(seed)
    x = torch.empty(tokens, experts, device="cuda").uniform_(-8, 0, generator=g)
    at = torch.randint(0, experts, (tokens, 1), device="cuda", generator=g)
    return x.scatter(1, at, torch.empty(tokens, 1, device="cuda").uniform_(4, 24, generator=g))


@pytest.mark.parametrize("experts,top_k", [(2, 1), (8, 2), (64, 8), (100, 12), (256, 32), (500, 4), (1000, 3)])
@pytest.mark.parametrize("renorm", [True, False])
def test_softmax_gradient_of_a_dominant_expert(experts, top_k, renorm):
    """One expert has nearly all the probability, so its gradient is what little the others take from it:
    c share_j sum_i share_i (d_j - d_i), or c p_j (d_j (1 - p_j) - sum_(i != j) d_i p_i) without
    renormalisation.  Bound: a probability's error, (16 + 2 range + E / 32) u as in the module's sums, twice,
    and k + 4 additions, of the sum of these terms' magnitudes."""
    fq = require_cuda()
    x = dominant(60, experts, experts + top_k)
    ids = fq.fp8q_moe_route(x, top_k, renormalize=renorm)["ids"].long()
    d = torch.randn(60, top_k, device="cuda", generator=gen(3))
    got = fq.fp8q_moe_route_backward(x, ids.int(), d, 0, renorm, 2.5).double()
    rel = (2 * (16 + 2 * float(x.max() - x.min()) + experts / 32) + top_k + 4) * U
    dd = d.double()
    if renorm:
        share = torch.softmax(x.double().gather(1, ids), 1)
        apart = dd[:, :, None] - dd[:, None, :]
        want = torch.zeros_like(x, dtype=torch.float64).scatter(1, ids, 2.5 * share * (share[:, None, :] * apart).sum(2))
        size = torch.zeros_like(want).scatter(1, ids, 2.5 * share * (share[:, None, :] * apart.abs()).sum(2))
    else:
        e = torch.exp(x.double() - x.double().amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        others = torch.stack([e[:, [j for j in range(experts) if j != i]].sum(1) for i in range(experts)], 1) / e.sum(1, keepdim=True)
        g = torch.zeros_like(p).scatter(1, ids, 2.5 * dd)
        dot, mag = (g * p).sum(1, keepdim=True), (g * p).abs().sum(1, keepdim=True)
        rest = torch.stack([torch.where(torch.arange(experts, device="cuda") == i, 0.0, g * p).sum(1) for i in ids.unique().tolist()], 1)
        mags = torch.stack([torch.where(torch.arange(experts, device="cuda") == i, 0.0, (g * p).abs()).sum(1) for i in ids.unique().tolist()], 1)
        col = {i: n for n, i in enumerate(ids.unique().tolist())}
        at = torch.tensor([col.get(i, 0) for i in range(experts)], device="cuda")
        chosen = torch.zeros_like(p, dtype=torch.bool).scatter(1, ids, True)
        want = p * torch.where(chosen, g * others - rest[:, at], -dot)
        size = p * torch.where(chosen, g.abs() * others + mags[:, at], mag)
    assert ((got - want).abs() <= rel * size + 1e-37).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
def test_weights_of_experts_that_a_bias_lifts_over_a_better_one(dtype, groups, top_groups):
    """A bias that chooses experts 90 to 130 below the best logit: the softmax over the chosen is what it is
    nearer the top, and agrees with its gradient.  Bound: (16 + 2 range) u, range that of the chosen."""
    fq = require_cuda()
    g = gen(4)
    x = torch.empty(40, 32, device="cuda").uniform_(-130, -90, generator=g)
    x[:, 31] = 0.0
    x = x.to(dtype)
    bias = torch.zeros(32, device="cuda")
    bias[:6] = torch.arange(9, 3, -1, device="cuda")
    r = fq.fp8q_moe_route(x, 4, 0, bias, groups, top_groups, weight_scale=2.5)
    assert (r["ids"] == torch.arange(4, device="cuda")).all()
    want = 2.5 * torch.softmax(x[:, :4].double(), 1)
    assert ((r["weights"].double() - want).abs() <= (16 + 2 * 40) * U * want + 1e-37).all()
    d = torch.randn(40, 4, device="cuda", generator=g)
    got = fq.fp8q_moe_route_backward(x, r["ids"], d, 0, True, 2.5)
    leaf = x.double().requires_grad_(True)
    (2.5 * torch.softmax(leaf[:, :4], 1) * d.double()).sum().backward()
    size = 2.5 * torch.softmax(x[:, :4].double(), 1) * d.double().abs().sum(1, keepdim=True)
    tol = 2 * (16 + 2 * 40 + 4) * U * size + leaf.grad[:, :4].abs() * (2.0 ** -8 if dtype == torch.bfloat16 else U)
    assert ((got[:, :4].double() - leaf.grad[:, :4]).abs() <= tol).all() and (got[:, 4:] == 0).all()


@pytest.mark.parametrize("experts,top_k", [(8, 2), (33, 4), (64, 8), (128, 6), (200, 5), (256, 8), (512, 16), (1000, 32), (1024, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_plain_softmax_gradient_of_every_expert(experts, top_k, dtype):
    """dx_e = c p_e (d_e [e chosen] - sum_j d_j p_j), each element to (2 (16 + 2 range + E / 32) + k) u of its own
    terms and the output's rounding.  The experts not chosen have gradients far above that bound, so that a
    kernel that leaves them out fails."""
    fq = require_cuda()
    x = torch.randn(65, experts, device="cuda", generator=gen(experts + top_k)).to(dtype)
    ids = fq.fp8q_moe_route(x, top_k, renormalize=False)["ids"]
    d = torch.randn(65, top_k, device="cuda", generator=gen(5))
    got = fq.fp8q_moe_route_backward(x, ids, d, 0, False, 2.5).double()
    p = torch.softmax(x.double(), 1)
    g = torch.zeros_like(p).scatter(1, ids.long(), 2.5 * d.double())
    want = p * (g - (g * p).sum(1, keepdim=True))
    size = p * (g.abs() + (g * p).abs().sum(1, keepdim=True))
    rel = (2 * (16 + 2 * float(x.float().max() - x.float().min()) + experts / 32) + top_k) * U
    tol = rel * size + (2.0 ** -8 if dtype == torch.bfloat16 else U) * want.abs()
    assert ((got - want).abs() <= tol).all()
    rest = torch.ones_like(p, dtype=torch.bool).scatter(1, ids.long(), False)
    assert (want[rest].norm() > 50 * tol[rest].norm()) and (got[rest] != 0).all()
