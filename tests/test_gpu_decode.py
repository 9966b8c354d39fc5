"""The expert layer for a few tokens against the layer in 64 bits.

Bounds, with u = 2^-24, on sums of magnitudes S = |W| |x|.  The tensor core adds 16 products to a sum at a
time and may cut what does not fit FP32: 4 u of the magnitudes each, 8 (16 with both parts of the inner
values) to a block of 128; blocks add in a row over at most 16 of a warp in these cases (or 64 in the second product),
8 warps, and take 4 roundings for scales: C1 = 32 + 16 + 8 + 4 and C2 = 64 + 64 + 8 + 4.  A token's values are off by 2^-39
of their group's largest, inner values by 2^-22 of themselves (2^-12 for BF16 output) and 2^-38 of their group's.  silu and its slope
(at most 1.1) pass the first product's error on, with 12 u of its own."""
import pytest
import torch

from gpu_util import Guarded, require_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
C1, C2 = 60, 140
TYPES = (torch.float8_e4m3fn, torch.float8_e5m2)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def weights(e, rows, cols, fmt, g):
    """Codes of every kind but NaN and Inf, and scales over several powers of two."""
    v = torch.randn(e, rows, cols, device="cuda", generator=g)
    q = (v * (100 if fmt == 0 else 3000)).clamp(-440, 440).to(TYPES[fmt]).view(torch.uint8)
    s = torch.exp2(torch.randint(-3, 4, (e, -(-rows // 128), -(-cols // 128)), device="cuda", generator=g).float())
    return q, s * (cols ** -0.5 / 100) * (1 + torch.rand(s.shape, device="cuda", generator=g))


def values(q, s, fmt):
    rows, cols = q.shape
    return q.view(TYPES[fmt]).double() * s.double().repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def layer64(x, ids, w, w1, s1, w2, s2, fmt, inner_half):
    """out and the bound of its error in FP32."""
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    xd, wd, n = x.double(), w.double(), w2.shape[2]
    for e in ids[(ids >= 0) & (ids < w1.shape[0])].unique().tolist():
        share = (wd * (ids == e)).sum(1, keepdim=True)
        size = (wd.abs() * (ids == e)).sum(1, keepdim=True)
        t = (ids == e).any(1)
        a1, a2 = values(w1[e], s1[e], fmt), values(w2[e], s2[e], fmt)
        h = xd[t] @ a1.T
        xm = xd[t].abs()
        h_err = C1 * U * (xm @ a1.abs().T) + 2.0 ** -39 * xm.amax(1, keepdim=True) * a1.abs().sum(1)
        gate, up = h.chunk(2, 1)
        g_err, u_err = h_err.chunk(2, 1)
        silu = gate * torch.sigmoid(gate)
        a = silu * up
        a_err = 1.1 * g_err * (up.abs() + u_err) + silu.abs() * u_err + (12 * U + inner_half) * a.abs() + 2.0 ** -38 * a.abs().amax(1, keepdim=True)
        y = a @ a2.T
        y_err = C2 * U * (a.abs() @ a2.abs().T) + a_err @ a2.abs().T
        out[t] += share[t] * y
        tol[t] += size[t] * (y_err + 40 * U * y.abs())
    return out, tol


def check(fq, x, ids, w, w1, s1, w2, s2, fmt, out_dtype=torch.float32):
    buf = Guarded(tuple(x.shape), out_dtype)
    got = fq.fp8q_moe_decode(x, ids, w, w1, s1, w2, s2, w_fmt=fmt, out_dtype=out_dtype, out=buf.t)
    want, tol = layer64(x, ids, w, w1, s1, w2, s2, fmt, 2.0 ** -22 if out_dtype == torch.float32 else 2.0 ** -12)
    bad = (got.double() - want).abs() > tol + HALF[out_dtype] * (want.abs() + tol) * (1 + 2.0 ** -7)
    assert not bad.any(), (int(bad.sum()), float((got.double() - want).abs().max()), float(want.abs().max()))
    buf.check()
    return got


def case(tokens, top, experts, hidden, inner, fmt, seed):
    g = gen(seed)
    x = torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16()
    ids = torch.rand(tokens, experts, device="cuda", generator=g).argsort(1)[:, :top].int().contiguous()
    w = torch.rand(tokens, top, device="cuda", generator=g)
    return [x, ids, w, *weights(experts, 2 * inner, hidden, fmt, g), *weights(experts, hidden, inner, fmt, g), fmt]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("tokens,top,experts,hidden,inner", [
    (1, 1, 1, 16, 16), (1, 8, 64, 1024, 256), (7, 3, 5, 272, 144), (8, 2, 2, 128, 128), (9, 1, 1, 2064, 80), (16, 8, 40, 512, 512),
    (33, 4, 300, 144, 272), (64, 6, 17, 1040, 336), (64, 32, 40, 256, 48), (64, 32, 1024, 32, 16), (5, 2, 1024, 32, 16), (48, 2, 3, 96, 2064)])
def test_layer(tokens, top, experts, hidden, inner, fmt):
    fq = require_cuda()
    for out_dtype in (torch.float32, torch.bfloat16):
        check(fq, *case(tokens, top, experts, hidden, inner, fmt, tokens + inner), out_dtype)


def test_full_width():
    """The measured layer's sizes, fewer experts."""
    fq = require_cuda()
    check(fq, *case(3, 4, 6, 7168, 2048, 0, 1))


def test_dropped_and_repeated_slots():
    fq = require_cuda()
    c = case(20, 4, 12, 256, 144, 0, 2)
    ids, w = c[1], c[2]
    ids[0] = -1                     # a token of no expert
    ids[1, 2], ids[2, 1] = -1, 99   # no expert's ids
    ids[3] = ids[3, 0]              # the same expert four times
    ids[4, 3] = ids[4, 1]
    w[5] = 0.0
    got = check(fq, *c)
    assert (got[0] == 0).all() and (got[5] == 0).all()
    ids.fill_(-1)
    assert (fq.fp8q_moe_decode(*c[:7], out_dtype=torch.bfloat16) == 0).all()
    ids.fill_(7)                    # every slot the same expert
    check(fq, *c)


def test_values_of_all_sizes():
    """Rows of zeros, tiny and huge rows, and large and small values in one group of 128."""
    fq = require_cuda()
    c = case(6, 2, 4, 384, 128, 0, 3)
    x = c[0]
    x[0] = 0
    x[1] *= 2.0 ** -60
    x[2] *= 2.0 ** 40
    x[3, ::2] *= 2.0 ** -20
    x[4, 5] = 2.0 ** 20
    check(fq, *c)


def test_nan_and_inf_stay_in_their_rows():
    fq = require_cuda()
    c = case(10, 2, 6, 256, 144, 0, 4)
    clean = fq.fp8q_moe_decode(*c[:7], out_dtype=torch.float32)
    x, ids, w = c[:3]
    x[2, 7], x[4, 100], w[6, 1] = float("nan"), float("inf"), float("nan")
    got = fq.fp8q_moe_decode(*c[:7], out_dtype=torch.float32)
    rest = [t for t in range(10) if t not in (2, 4, 6)]
    assert torch.isnan(got[2]).all() and torch.isnan(got[6]).all() and not torch.isfinite(got[4]).any()
    assert torch.equal(got[rest], clean[rest])
    c = case(10, 2, 6, 256, 144, 0, 4)
    c[3][1, 20, 30] = 0x7F          # a NaN weight: the tokens of its expert
    got = fq.fp8q_moe_decode(*c[:7], out_dtype=torch.float32)
    hit = (c[1] == 1).any(1)
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])


def test_large_offsets():
    """Weights past 2^31 bytes."""
    fq = require_cuda()
    e, hidden, inner = 160, 4096, 2048
    g = gen(5)
    w1 = torch.randint(0, 120, (e, 2 * inner, hidden), dtype=torch.uint8, device="cuda", generator=g)
    w2 = torch.randint(0, 120, (e, hidden, inner), dtype=torch.uint8, device="cuda", generator=g)
    assert w1.numel() > 2 ** 31
    s1, s2 = torch.full((e, 32, 32), 1e-3, device="cuda"), torch.full((e, 32, 16), 1e-3, device="cuda")
    x = torch.randn(2, hidden, device="cuda", generator=g).bfloat16()
    ids = torch.tensor([[159, 150], [0, 158]], dtype=torch.int32, device="cuda")
    check(fq, x, ids, torch.rand(2, 2, device="cuda", generator=g), w1, s1, w2, s2, 0)


def test_same_bits_on_streams_and_in_graphs():
    fq = require_cuda()
    c = case(12, 4, 16, 512, 272, 0, 6)
    want = fq.fp8q_moe_decode(*c[:7])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = [fq.fp8q_moe_decode(*c[:7]) for _ in range(5)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = fq.fp8q_moe_decode(*c[:7])
    for i in range(3):
        d = case(12, 4, 16, 512, 272, 0, 20 + i)
        for a, b in zip(c[:7], d[:7]):
            a.copy_(b)
        graph.replay()
        assert torch.equal(held, fq.fp8q_moe_decode(*d[:7]))


def test_after_routing():
    """The routing's weights and ids as they are, and the grouped path's result within its own rounding: each
    of that path's products of E4M3 copies is off by sqrt(2^-8 + 2^-8) in the norm at most, twice through the gate."""
    fq = require_cuda()
    x, _, _, w1, s1, w2, s2, _ = case(24, 1, 8, 512, 256, 0, 7)
    logits = torch.randn(24, 8, device="cuda", generator=gen(8))
    r = fq.fp8q_moe_route(logits, 2)
    got = check(fq, x, r["ids"], r["weights"], w1, s1, w2, s2, 0)
    plan = fq.fp8q_moe_plan(r["ids"], 8)
    q = fq.fp8q_moe_dispatch(x, plan)
    h = fq.fp8q_matmul_grouped(q["q"], q["scale_inv"], w1, s1, plan["offsets"])
    a = fq.fp8q_swiglu(h)
    y = fq.fp8q_matmul_grouped(a["q"], a["scale_inv"], w2, s2, plan["offsets"])
    other = fq.fp8q_moe_combine(y, plan, r["weights"]).float()
    off = 2.0 ** -3.5
    assert (other - got).norm() <= (3 * off + 2.0 ** -6) * got.norm()


def test_refusals():
    fq = require_cuda()
    x, ids, w, w1, s1, w2, s2, _ = case(4, 2, 3, 64, 32, 0, 9)
    for bad in ((x.float(), ids, w, w1, s1, w2, s2), (x, ids.long(), w, w1, s1, w2, s2), (x, ids, w[:2], w1, s1, w2, s2),
                (x, ids[:2], w[:2], w1, s1, w2, s2), (x, ids, w, w1[:2], s1, w2, s2), (x, ids, w, w1, s1[:, :, :0], w2, s2),
                (x, ids, w, w1, s1, w2, s2.cpu()), (x[:, :32], ids, w, w1, s1, w2, s2), (x.cpu(), ids, w, w1, s1, w2, s2),
                (x, ids, w, w1.view(torch.int8), s1, w2, s2)):
        with pytest.raises(ValueError):
            fq.fp8q_moe_decode(*bad)
    with pytest.raises(fq.Fp8qError, match="64 tokens"):
        fq.fp8q_moe_decode(x.repeat(17, 1), ids.repeat(17, 1), w.repeat(17, 1), w1, s1, w2, s2)
    assert fq.fp8q_moe_decode(x[:0], ids[:0], w[:0], w1, s1, w2, s2).shape == (0, 64)
