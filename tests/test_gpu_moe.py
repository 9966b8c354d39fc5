"""The expert layer: routing, row order, gather and quantize, weighted sum, and
their gradients, against plain restatements in 64 bits.

Tolerances, with u = 2^-23.  A score is an exponential (2 units, and its argument x - max is
rounded: |x - max| units more), a sum of E of them (E / 32 + 5 additions in a row) and divisions
and products of half a unit each: rel = (16 + 2 range + E / 32) u covers a weight, twice that
one factor of a gradient.  Sums over j or over columns add (terms) u of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import Guarded, dev, host, require_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
NEG = float("-inf")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
def keys64(x, score, bias, groups, top_groups):
    """Scores and keys in 64 bits, keys of what cannot be chosen at -inf."""
    x = x.double()
    s = torch.softmax(x, 1) if score == 0 else 1 / (1 + torch.exp(-x))
    k = x.clone() if bias is None and groups == 1 else s + (0 if bias is None else bias.double())
    k[~(x > NEG)] = NEG
    k[~(k > NEG)] = NEG
    group_worth = None
    if groups > 1:
        best = k.view(x.shape[0], groups, -1).sort(2, descending=True).values
        group_worth = best[:, :, :2].sum(2)
    return s, k, group_worth


def check_route(r, x, top_k, score, bias=None, groups=1, top_groups=1, renorm=True, scale=1.0):
    t, e = x.shape
    s, k, worth = keys64(x, score, bias, groups, top_groups)
    spread = float((x.float().max() - x.float()[x.float() > NEG].min()).clamp_max(200)) if (x.float() > NEG).any() else 0
    rel = (16 + 2 * spread + e / 32) * U
    tol = rel * 4 if not (bias is None and groups == 1) else 0.0
    ids, w = r["ids"].long(), r["weights"].double()
    if groups > 1:  # every chosen expert's group is worth as much as the top_groups-th best
        limit = worth.sort(1, descending=True).values[:, top_groups - 1:top_groups]
        of = (ids.clamp_min(0) // (e // groups))
        got = worth.gather(1, of)
        assert ((got >= limit - tol) | (ids < 0)).all()
        assert all(len(set(row)) <= top_groups for row in torch.where(ids >= 0, of, of[:, :1]).tolist())
        allowed = torch.zeros(t, groups, dtype=torch.bool, device="cuda")
        rank = worth.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
        allowed.scatter_(1, rank, True)
        clear = (worth.sort(1, descending=True).values[:, top_groups - 1] -
                 (worth.sort(1, descending=True).values[:, top_groups] if top_groups < groups else NEG)) > tol
        k = torch.where(allowed.repeat_interleave(e // groups, 1), k, NEG)
    else:
        clear = torch.ones(t, dtype=torch.bool, device="cuda")
    for row in ids.tolist():
        real = [i for i in row if i >= 0]
        assert len(set(real)) == len(real) and all(0 <= i < e for i in real)
        assert row[:len(real)] == real  # -1 only at the end
    best = k.sort(1, descending=True).values[:, :top_k]
    mine = k.gather(1, ids.clamp_min(0))
    fits = torch.where(ids >= 0, (mine - best).abs() <= tol, best == NEG)
    assert fits[clear].all()
    chosen = s.gather(1, ids.clamp_min(0)) * (ids >= 0)
    want = scale * (chosen / chosen.sum(1, keepdim=True).clamp_min(1e-300) if renorm else chosen)
    assert ((w - want).abs() <= rel * want.abs() + 1e-37).all()


@pytest.mark.parametrize("experts", [1, 2, 7, 32, 33, 64, 100, 160, 256, 257, 512, 1000, 1024])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_sizes(experts, score, dtype):
    fq = require_cuda()
    g = gen(experts)
    for tokens, top_k in ((1, 1), (37, min(8, experts)), (9, min(32, experts))):
        x = torch.randn(tokens, experts, device="cuda", generator=g).to(dtype)
        bias = 0.3 * torch.randn(experts, device="cuda", generator=g)
        for b in (None, bias):
            for renorm in (True, False):
                r = fq.fp8q_moe_route(x, top_k, score, b, renormalize=renorm, weight_scale=2.5)
                check_route(r, x, top_k, score, b, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("experts,groups,top_groups,top_k", [(64, 8, 4, 8), (256, 8, 4, 8), (160, 8, 3, 6), (30, 3, 2, 4),
                                                             (32, 32, 5, 5), (100, 5, 5, 7), (1024, 16, 1, 32), (12, 6, 1, 2)])
@pytest.mark.parametrize("score", [0, 1])
def test_route_groups(experts, groups, top_groups, top_k, score):
    fq = require_cuda()
    g = gen(experts + groups)
    x = torch.randn(300, experts, device="cuda", generator=g)
    bias = 0.1 * torch.randn(experts, device="cuda", generator=g)
    for b in (None, bias):
        r = fq.fp8q_moe_route(x, top_k, score, b, groups, top_groups)
        check_route(r, x, top_k, score, b, groups, top_groups)


def test_route_ties_go_to_the_lowest_index():
    fq = require_cuda()
    x = torch.zeros(3, 100, device="cuda")
    x[1] = torch.tensor([1.0, -0.0, 0.0, 2.0] * 25, device="cuda")
    x[2, 50:] = 1.0
    r = fq.fp8q_moe_route(x, 6)
    assert r["ids"].tolist() == [[0, 1, 2, 3, 4, 5], [3, 7, 11, 15, 19, 23], [50, 51, 52, 53, 54, 55]]
    r = fq.fp8q_moe_route(x, 6, fq.SCORE_SIGMOID, torch.zeros(100, device="cuda"), 10, 2)
    assert r["ids"].tolist() == [[0, 1, 2, 3, 4, 5], [3, 7, 11, 15, 19, 0], [50, 51, 52, 53, 54, 55]]


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_masked_logits(score, renorm):
    """-inf leaves 0, 1, 2 or all experts; the lowest finite value is an ordinary logit; NaN poisons the weights."""
    fq = require_cuda()
    g = gen(5)
    x = torch.randn(6, 40, device="cuda", generator=g)
    x[0] = NEG
    x[1] = NEG
    x[1, 17] = 0.5
    x[2] = NEG
    x[2, 3], x[2, 39] = -1.0, 2.0
    x[3] = torch.finfo(torch.float32).min
    x[4, 11] = float("nan")
    x[4, 20] = 9.0
    for bias in (None, torch.zeros(40, device="cuda")):
        r = fq.fp8q_moe_route(x, 3, score, bias, renormalize=renorm)
        ids, w = r["ids"].tolist(), r["weights"]
        assert ids[0] == [-1, -1, -1] and w[0].tolist() == [0, 0, 0]
        assert ids[1] == [17, -1, -1] and w[1, 1:].tolist() == [0, 0]
        assert w[1, 0].item() == pytest.approx(1.0 if renorm or score == 0 else 1 / (1 + np.exp(-0.5)), rel=4 * U)
        assert ids[2] == [39, 3, -1] and w[2, 2].item() == 0
        assert ids[3] == [0, 1, 2]
        if score == 0:  # equal logits
            assert w[3].tolist() == pytest.approx([1 / 3 if renorm else 1 / 40] * 3, rel=64 * U)
        else:  # scores of exactly 0
            assert w[3].tolist() == [0, 0, 0]
        assert ids[4][0] == 20 and 11 not in ids[4] and torch.isnan(w[4]).all()
        assert torch.isfinite(w[5]).all()
        ok = x[1:3]
        check_route({k: v[1:3] for k, v in r.items()}, ok, 3, score, bias, renorm=renorm)
    x[4, 11] = float("inf")
    r = fq.fp8q_moe_route(x, 3, score, renormalize=renorm)
    assert r["ids"][4, 0].item() == 11 and torch.isnan(r["weights"][4]).all() == (score == 0)
    bias = torch.zeros(40, device="cuda")
    bias[5:] = NEG  # a mask for all tokens
    r = fq.fp8q_moe_route(x[5:], 8, score, bias, renormalize=renorm)
    assert sorted(r["ids"][0, :5].tolist()) == [0, 1, 2, 3, 4] and r["ids"][0, 5:].tolist() == [-1] * 3


def test_route_large_logits():
    """Differences that overflow or underflow an exponential without the maximum taken off."""
    fq = require_cuda()
    x = torch.tensor([[3e38, -3e38, 0.0, 3e38], [-3e38, -2e38, -1e38, -3e38], [200.0, 199.0, -200.0, 0.0]], device="cuda")
    r = fq.fp8q_moe_route(x, 2)
    assert r["ids"].tolist() == [[0, 3], [2, 1], [0, 1]]
    assert r["weights"].tolist() == [[0.5, 0.5], [1.0, 0.0], pytest.approx([1 / (1 + np.exp(-1)), 1 / (1 + np.e)], rel=16 * U)]


def route64(x, ids, score, renorm, scale):
    s = torch.softmax(x, 1) if score == 0 else torch.sigmoid(x)
    c = s.gather(1, ids.clamp_min(0)) * (ids >= 0)
    return scale * (c / c.sum(1, keepdim=True) if renorm else c)


@pytest.mark.parametrize("experts,top_k", [(1, 1), (8, 2), (64, 8), (100, 6), (256, 8), (1000, 32)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_backward(experts, top_k, score, renorm, dtype):
    fq = require_cuda()
    g = gen(experts + top_k)
    x = torch.randn(65, experts, device="cuda", generator=g).to(dtype)
    r = fq.fp8q_moe_route(x, top_k, score, renormalize=renorm, weight_scale=2.5)
    d = torch.randn(65, top_k, device="cuda", generator=g)
    got = fq.fp8q_moe_route_backward(x, r["ids"], d, score, renorm, 2.5)
    assert got.dtype == dtype
    leaf = x.double().requires_grad_(True)
    w = route64(leaf, r["ids"].long(), score, renorm, 2.5)
    w.backward(d.double())
    spread = float(x.float().max() - x.float().min())
    # terms of one element: 2.5 |s_j| (|d_j| + mean |d|) at most, each with a weight's error, twice
    size = 2.5 * d.double().abs().sum(1, keepdim=True)
    tol = 2 * (16 + 2 * spread + experts / 32 + top_k) * U * size + leaf.grad.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else U)
    assert ((got.double() - leaf.grad).abs() <= tol).all()
    # central differences of the 64-bit forward along a random direction: error of order h^2
    v = torch.randn(65, experts, dtype=torch.float64, device="cuda", generator=g)
    h = 1e-4
    up, dn = (route64(x.double() + a * v, r["ids"].long(), score, renorm, 2.5) for a in (h, -h))
    slope = ((up - dn) / (2 * h) * d.double()).sum(1)
    mine = (got.double() * v).sum(1)
    assert ((mine - slope).abs() <= (tol * v.abs()).sum(1) + 100 * h * h * size[:, 0] * v.abs().amax(1) ** 3).all()


def test_route_backward_of_dropped_slots():
    fq = require_cuda()
    x = torch.full((2, 20), NEG, device="cuda")
    x[1, 4], x[1, 9] = 1.0, 2.0
    for score in (0, 1):
        for renorm in (True, False):
            r = fq.fp8q_moe_route(x, 3, score, renormalize=renorm)
            got = fq.fp8q_moe_route_backward(x, r["ids"], torch.ones(2, 3, device="cuda") * torch.tensor([1., 2., 3.], device="cuda"), score, renorm)
            leaf = x[1:, [9, 4]].double().requires_grad_(True)
            (route64(leaf, torch.tensor([[0, 1]], device="cuda"), score, renorm, 1.0) * torch.tensor([1., 2.], device="cuda")).sum().backward()
            assert (got[0] == 0).all()
            assert torch.allclose(got[1, [9, 4]].double(), leaf.grad[0], rtol=0, atol=100 * U)
            rest = torch.ones(20, dtype=torch.bool)
            rest[[4, 9]] = False
            assert (got[1, rest.cuda()] == 0).all()


def test_route_writes_inside_its_outputs():
    fq = require_cuda()
    x = torch.randn(77, 50, device="cuda", generator=gen(1))
    w, i, d = Guarded((77, 5), torch.float32), Guarded((77, 5), torch.int32), Guarded((77, 50), torch.float32)
    fq.fp8q_moe_route(x, 5, out={"weights": w.t, "ids": i.t})
    fq.fp8q_moe_route_backward(x, i.t, w.t, out=d.t)
    torch.cuda.synchronize()
    for b in (w, i, d):
        b.check()
    assert fq.fp8q_moe_route(x[:0], 5)["ids"].shape == (0, 5)


# ---------------------------------------------------------------------------
# row order
# ---------------------------------------------------------------------------
def plan_reference(ids, experts, align, rows):
    flat = ids.reshape(-1)
    row_of = np.full(flat.size, -1, np.int32)
    src = np.full(rows, -1, np.int32)
    offsets, at = [0], 0
    for e in range(experts):
        mine = np.flatnonzero(flat == e)
        row_of[mine] = at + np.arange(mine.size)
        src[at:at + mine.size] = mine
        at += -(-mine.size // align) * align
        offsets.append(at)
    return np.array(offsets), row_of.reshape(ids.shape), src


@pytest.mark.parametrize("tokens,top_k,experts", [(0, 2, 5), (1, 1, 1), (1, 8, 64), (16, 8, 64), (333, 3, 7), (1000, 8, 256), (511, 8, 1024),
                                                  (512, 8, 100), (4097, 1, 33), (3000, 8, 64), (70000, 2, 60)])
@pytest.mark.parametrize("align", [1, 16, 128])
def test_plan(tokens, top_k, experts, align):
    fq = require_cuda()
    rng = np.random.default_rng(tokens + experts)
    ids = rng.integers(0, experts, (tokens, top_k)).astype(np.int32)
    if experts > 3:
        ids[ids == 2] = 3  # an expert nobody wants
    drop = rng.random(ids.shape) < 0.05
    ids[drop] = rng.choice(np.array([-1, -7, experts, 2 ** 31 - 1], np.int32), int(drop.sum()))
    rows = fq.fp8q_moe_rows(ids.size, experts, align)
    out = {"offsets": Guarded((experts + 1,), torch.int64), "row_of": Guarded(ids.shape, torch.int32), "src": Guarded((rows,), torch.int32)}
    p = fq.fp8q_moe_plan(dev(ids), experts, align, out={k: v.t for k, v in out.items()})
    torch.cuda.synchronize()
    valid = np.where((ids >= 0) & (ids < experts), ids, -1)
    offsets, row_of, src = plan_reference(valid, experts, align, rows)
    np.testing.assert_array_equal(p["offsets"].cpu().numpy(), offsets)
    np.testing.assert_array_equal(p["row_of"].cpu().numpy(), row_of)
    np.testing.assert_array_equal(p["src"].cpu().numpy(), src)
    for b in out.values():
        b.check()


def test_plan_of_one_expert_and_of_no_slot():
    fq = require_cuda()
    ids = np.full((5000, 4), 17, np.int32)
    p = fq.fp8q_moe_plan(dev(ids), 64, 128)
    offsets, row_of, src = plan_reference(ids, 64, 128, p["src"].numel())
    np.testing.assert_array_equal(p["row_of"].cpu().numpy(), row_of)
    np.testing.assert_array_equal(p["src"].cpu().numpy(), src)
    p = fq.fp8q_moe_plan(dev(np.full((40, 4), -1, np.int32)), 64, 128)
    assert (p["offsets"] == 0).all() and (p["row_of"] == -1).all() and (p["src"] == -1).all()


# ---------------------------------------------------------------------------
# gather and quantize
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,top_k,experts,cols", [(1, 1, 2, 16), (1, 8, 64, 144), (37, 3, 5, 400), (200, 2, 9, 256), (150, 8, 16, 1040)])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("pow2", [False, True])
def test_dispatch_equals_quantizing_the_gathered_rows(tokens, top_k, experts, cols, fmt, pow2):
    fq = require_cuda()
    g = gen(tokens + cols)
    x = (torch.randn(tokens, cols, device="cuda", generator=g) * torch.exp2(8 * torch.randn(tokens, 1, device="cuda", generator=g))).bfloat16()
    x[tokens // 2, 3] = float("inf")
    x[0, 7] = float("nan")
    ids = torch.randint(-1, experts, (tokens, top_k), generator=g, device="cuda").int()
    for align, direction in ((1, fq.ROW), (128, fq.BOTH), (16, fq.COL)):
        p = fq.fp8q_moe_plan(ids, experts, align)
        rows = p["src"].numel()
        src = p["src"].long()
        xg = torch.where((src >= 0)[:, None], x[src.clamp_min(0) // top_k], torch.zeros_like(x[:1]))
        out = {"q": Guarded((rows, cols)), "q_t": Guarded((cols, rows)), "scale_inv": Guarded((rows, -(-cols // 128)), torch.float32),
               "scale_inv_t": Guarded((cols, -(-rows // 128)), torch.float32)}
        r = fq.fp8q_moe_dispatch(x, p, fmt, direction, pow2, out={k: v.t for k, v in out.items()})
        bits = host(xg.view(torch.int16)).view(np.uint16)
        if direction & fq.ROW:
            q, si = oracle.blockwise(bits, fmt, (1, 128), pow2)
            np.testing.assert_array_equal(host(r["q"]), q)
            np.testing.assert_array_equal(host(r["scale_inv"]).view(np.uint32), si.view(np.uint32))
        if direction & fq.COL:
            q, si = oracle.blockwise(bits, fmt, (128, 1), pow2)
            np.testing.assert_array_equal(host(r["q_t"]), q.T)
            np.testing.assert_array_equal(host(r["scale_inv_t"]).view(np.uint32), np.ascontiguousarray(si.T).view(np.uint32))
        for b in out.values():
            b.check()


def test_dispatch_of_a_large_batch_equals_the_quantizer():
    fq = require_cuda()
    g = gen(3)
    x = torch.randn(4000, 7168, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, 64, (4000, 8), generator=g, device="cuda").int()
    p = fq.fp8q_moe_plan(ids, 64, 128)
    src = p["src"].long()
    xg = torch.where((src >= 0)[:, None], x[src.clamp_min(0) // 8], torch.zeros_like(x[:1]))
    r, w = fq.fp8q_moe_dispatch(x, p, direction=fq.BOTH), fq.fp8q_quantize_blockwise(xg, direction=fq.BOTH)
    for k in r:
        assert torch.equal(r[k], w[k]), k


@pytest.mark.parametrize("rows", [1, 17, 129])
def test_rowwise_quantizer_takes_any_rows(rows):
    """The quantizer's rowwise copy of a decode batch, which has no multiple of 16 rows."""
    fq = require_cuda()
    x = torch.randn(rows, 400, device="cuda", generator=gen(rows)).bfloat16()
    for block in (fq.BLOCK_1X128, fq.BLOCK_128X128):
        out = {"q": Guarded((rows, 400)), "scale_inv": Guarded((rows if block == 1 else -(-rows // 128), 4), torch.float32)}
        r = fq.fp8q_quantize_blockwise(x, block=block, out={k: v.t for k, v in out.items()})
        q, si = oracle.blockwise(host(x.view(torch.int16)).view(np.uint16), 0, (1, 128) if block == 1 else (128, 128))
        np.testing.assert_array_equal(host(r["q"]), q)
        np.testing.assert_array_equal(host(r["scale_inv"]), si)
        for b in out.values():
            b.check()


# ---------------------------------------------------------------------------
# weighted sum
# ---------------------------------------------------------------------------
def half_unit(v, dtype):
    return v.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else U) + 1e-38


@pytest.mark.parametrize("tokens,top_k,experts,cols", [(1, 1, 1, 1), (1, 8, 64, 7168), (7, 2, 5, 33), (60, 8, 16, 264), (129, 3, 4, 1024),
                                                       (40, 32, 40, 520)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("align", [1, 128])
def test_combine_and_its_gradients(tokens, top_k, experts, cols, dtype, align):
    fq = require_cuda()
    g = gen(tokens + cols)
    ids = torch.randint(-1 if tokens > 1 else 0, experts, (tokens, top_k), generator=g, device="cuda").int()
    p = fq.fp8q_moe_plan(ids, experts, align)
    rows = p["src"].numel()
    y = torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
    y[p["src"] < 0] = float("nan")  # padding is never read
    w = torch.randn(tokens, top_k, device="cuda", generator=g)
    w[ids < 0] = float("nan")       # nor are the weights of dropped slots
    d = torch.randn(tokens, cols, device="cuda", generator=g).to(dtype)
    at, there = p["row_of"].long().clamp_min(0), (p["row_of"] >= 0)
    yv = torch.where(there[:, :, None], y.double()[at], 0.0)
    wv = torch.where(there, w.double(), 0.0)
    out = Guarded((tokens, cols), dtype)
    fq.fp8q_moe_combine(y, p, w, out=out.t)
    want, size = (yv * wv[:, :, None]).sum(1), (yv * wv[:, :, None]).abs().sum(1)
    assert ((out.t.double() - want).abs() <= top_k * U * size + half_unit(want, dtype)).all()
    out.check()
    fq.fp8q_moe_combine(y, p, out=out.t)
    want, size = yv.sum(1), yv.abs().sum(1)
    assert ((out.t.double() - want).abs() <= top_k * U * size + half_unit(want, dtype)).all()
    bufs = {"d_y": Guarded((rows, cols), dtype), "d_weights": Guarded((tokens, top_k), torch.float32)}
    r = fq.fp8q_moe_combine_backward(d, y, p, w, out={k: v.t for k, v in bufs.items()})
    want = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    src = p["src"].long()
    real = src >= 0
    want[real] = wv.reshape(-1)[src[real]][:, None] * d.double()[src[real] // top_k]
    assert ((r["d_y"].double() - want).abs() <= half_unit(want, dtype)).all() and (r["d_y"][~real] == 0).all()
    prod = yv * d.double()[:, None, :]
    assert ((r["d_weights"].double() - prod.sum(2)).abs() <= (cols / 64 + 16) * U * prod.abs().sum(2)).all()
    for b in bufs.values():
        b.check()


def test_combine_gradients_against_differences():
    """The 64-bit sum is linear in y and in w: its differences are its gradients."""
    fq = require_cuda()
    g = gen(9)
    ids = torch.randint(0, 6, (20, 3), generator=g, device="cuda").int()
    p = fq.fp8q_moe_plan(ids, 6, 16)
    rows = p["src"].numel()
    y, vy = (torch.randn(rows, 48, device="cuda", generator=g) for _ in range(2))
    w, vw = (torch.randn(20, 3, device="cuda", generator=g) for _ in range(2))
    d = torch.randn(20, 48, device="cuda", generator=g)
    vy[p["src"] < 0] = 0

    def f(y, w):
        return (y[p["row_of"].long()] * w[:, :, None]).sum(1)

    r = fq.fp8q_moe_combine_backward(d, y, p, w)
    for got, slope, size in (((r["d_y"].double() * vy).sum(), (f((y + vy).double(), w.double()) - f((y - vy).double(), w.double())) / 2, vy.abs().sum()),
                             ((r["d_weights"].double() * vw).sum(), (f(y.double(), (w + vw).double()) - f(y.double(), (w - vw).double())) / 2, vw.abs().sum())):
        want = (slope * d.double()).sum()
        # one rounding of y + v (and w + v) and of each gradient, at most 8 in size, over 60 x 48 terms
        assert abs(got - want) <= 64 * 8 * U * (size + (slope.abs() * d.abs()).sum())


def test_combine_misaligned_rows():
    """A y that starts 2 bytes off takes the element loads."""
    fq = require_cuda()
    g = gen(10)
    ids = torch.randint(0, 4, (9, 2), generator=g, device="cuda").int()
    p = fq.fp8q_moe_plan(ids, 4)
    raw = torch.randn(18 * 64 + 1, device="cuda", generator=g).bfloat16()
    y = raw[1:].view(18, 64)
    w = torch.rand(9, 2, device="cuda", generator=g)
    assert torch.equal(fq.fp8q_moe_combine(y, p, w), fq.fp8q_moe_combine(y.clone(), p, w))
    d = torch.randn(9, 64, device="cuda", generator=g).bfloat16()
    a, b = fq.fp8q_moe_combine_backward(d, y, p, w), fq.fp8q_moe_combine_backward(d, y.clone(), p, w)
    assert torch.equal(a["d_y"], b["d_y"])
    assert torch.allclose(a["d_weights"], b["d_weights"], rtol=0, atol=64 * 64 * U)


def test_rows_beyond_31_bits_of_elements():
    """Rows whose elements lie past 2^31: the dispatch and the sum address them in 64 bits."""
    fq = require_cuda()
    g = gen(11)
    tokens, top_k, cols = 40000, 8, 7168
    x = torch.randn(tokens, cols, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, 16, (tokens, top_k), generator=g, device="cuda").int()
    p = fq.fp8q_moe_plan(ids, 16, 1)
    r = fq.fp8q_moe_dispatch(x, p)
    at = torch.tensor([0, 299593, 299594, 319999], device="cuda")
    w = fq.fp8q_quantize_blockwise(x[p["src"][at].long() // top_k])
    assert torch.equal(r["q"][at], w["q"]) and torch.equal(r["scale_inv"][at], w["scale_inv"])
    del r
    y = x.repeat(8, 1)
    out = fq.fp8q_moe_combine(y, p)
    t = torch.tensor([0, 1, 39999], device="cuda")
    want = y[p["row_of"][t].long()].double().sum(1)
    assert ((out[t].double() - want).abs() <= 8 * U * y[p["row_of"][t].long()].double().abs().sum(1) + half_unit(want, torch.bfloat16)).all()


def test_on_another_stream():
    fq = require_cuda()
    g = gen(12)
    x = torch.randn(500, 512, device="cuda", generator=g).bfloat16()
    logits = torch.randn(500, 32, device="cuda", generator=g)

    def path():
        r = fq.fp8q_moe_route(logits, 4)
        p = fq.fp8q_moe_plan(r["ids"], 32, 128)
        q = fq.fp8q_moe_dispatch(x, p, direction=fq.BOTH)
        return [r["weights"], p["src"], q["q"], q["q_t"], fq.fp8q_moe_combine(torch.ones(p["src"].numel(), 512, device="cuda"), p, r["weights"])]

    want = path()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = path()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_python_checks():
    fq = require_cuda()
    x = torch.zeros(4, 32, device="cuda")
    b = torch.zeros(4, 32, device="cuda", dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    p = fq.fp8q_moe_plan(ids, 8)
    for bad in (lambda: fq.fp8q_moe_route(x.cpu(), 2), lambda: fq.fp8q_moe_route(x.t(), 2), lambda: fq.fp8q_moe_route(x.half(), 2),
                lambda: fq.fp8q_moe_route(x, 2, bias=torch.zeros(31, device="cuda")), lambda: fq.fp8q_moe_route_backward(x, ids[:3], w[:3]),
                lambda: fq.fp8q_moe_route_backward(x, ids, w[:, :1].contiguous()), lambda: fq.fp8q_moe_plan(ids.long(), 8),
                lambda: fq.fp8q_moe_plan(ids, 0), lambda: fq.fp8q_moe_dispatch(x, p), lambda: fq.fp8q_moe_dispatch(b[:3], p),
                lambda: fq.fp8q_moe_combine(x.t(), p, w), lambda: fq.fp8q_moe_combine(torch.zeros(8, 32, device="cuda"), p, w[:2]),
                lambda: fq.fp8q_moe_combine_backward(x, b, p, w), lambda: fq.fp8q_moe_combine_backward(x, torch.zeros(9, 32, device="cuda"), p, w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fq.fp8q_moe_route(x, 33), lambda: fq.fp8q_moe_route(x, 2, num_groups=5), lambda: fq.fp8q_moe_route(x, 9, num_groups=4),
                lambda: fq.fp8q_moe_dispatch(b[:, :24].contiguous(), p), lambda: fq.fp8q_moe_dispatch(b, p, direction=fq.BOTH),
                lambda: fq.fp8q_moe_plan(ids, 1025)):
        with pytest.raises(fq.Fp8qError):
            bad()


def test_a_plan_that_is_not_one_is_refused():
    fq = require_cuda()
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    p = fq.fp8q_moe_plan(ids, 8)
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    y, w = torch.zeros(8, 128, device="cuda"), torch.zeros(4, 2, device="cuda")
    d = torch.zeros(4, 128, device="cuda")
    for bad in (dict(p, src=p["src"].long()), dict(p, src=p["src"].cpu()), dict(p, src=p["src"].repeat(2)[::2]),
                dict(p, src=p["src"].view(2, 4)), dict(p, row_of=p["row_of"].long()), dict(p, row_of=p["row_of"].cpu())):
        for call in (lambda: fq.fp8q_moe_dispatch(x, bad), lambda: fq.fp8q_moe_combine_backward(d, y, bad, w)):
            with pytest.raises(ValueError):
                call()
