"""The norm and the gated activation, their copies and gradients, against plain restatements in 64 bits.

Tolerances, with u = 2^-24 (half a step of FP32 relative to the value).  A row's sum of squares or of
products adds at most 32 values a thread, 5 between lanes and 32 between warps: SUM = 70 roundings of
terms of one sign (or of the sum of magnitudes).  rstd takes half of it, half of 1 / columns, a product
and an addition, and two units (4 u) of the reciprocal root: under 41 u.  y takes two products more.  A code is off by half a step of its type
(eps / 2 relative to the value, or half the smallest step times the scale below the normal range)."""
import numpy as np
import pytest
import torch

from gpu_util import Guarded, require_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SUM = 70
BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, FP32: U}
TYPES = (torch.float8_e4m3fn, torch.float8_e5m2)
CODE_HALF = (2.0 ** -4, 2.0 ** -3)
CODE_SUB = (2.0 ** -10, 2.0 ** -17)
LARGEST = (448.0, 57344.0)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def near(got, want, tol):
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.numel(), float((got.double() - want).abs()[bad].max()))


def check_copy(q, inv, want, fmt, rel, pow2=False):
    """q, inv: codes in groups of 128 along the rows of `want` (64 bits), whose values are known to `rel`."""
    rows, cols = want.shape
    assert q.shape == (rows, cols) and inv.shape == (rows, -(-cols // 128))
    pad = torch.zeros(rows, inv.shape[1] * 128, dtype=torch.float64, device="cuda")
    pad[:, :cols] = want.abs()
    amax = pad.view(rows, -1, 128).amax(2)
    scale = 1 / inv.double()
    if pow2:
        assert (torch.frexp(inv)[0] == 0.5).all()
        top = amax * scale
        assert ((top <= LARGEST[fmt] * (1 + rel + 4 * U)) | (amax == 0)).all() and ((top * 2 >= LARGEST[fmt] * (1 - rel - 4 * U)) | (amax == 0)).all()
    else:
        near(inv, torch.where(amax > 0, amax / LARGEST[fmt], torch.ones_like(amax)), amax / LARGEST[fmt] * (rel + 4 * U))
    wide = inv.double().repeat_interleave(128, 1)[:, :cols]
    got = q.view(TYPES[fmt]).double() * wide
    near(got, want, want.abs() * (CODE_HALF[fmt] * (1 + 2 * rel + 8 * U) + rel + 8 * U) + CODE_SUB[fmt] * wide)


def codes_of(v, fmt, pow2=False):
    """The blockwise quantizer's rule for FP32 values v (groups of 128 along the rows), step by step in numpy."""
    v = v.cpu().numpy()
    rows, cols = v.shape
    pad = np.zeros((rows, -(-cols // 128) * 128), np.float32)
    pad[:, :cols] = np.abs(v)
    amax = pad.reshape(rows, -1, 128).max(2)  # NaN wins
    with np.errstate(all="ignore"):
        scale = np.minimum(np.float32(LARGEST[fmt]) / amax, np.float32(3.4028235e38))
        scale[~np.isfinite(amax) | (amax == 0)] = 1
        if pow2:
            scale = (scale.view(np.uint32) & np.uint32(0xFF800000)).view(np.float32)
        scaled = v * np.repeat(scale, 128, 1)[:, :cols]
    t = torch.from_numpy(scaled).clamp(-LARGEST[fmt], LARGEST[fmt]).to(TYPES[fmt]).view(torch.uint8).numpy().copy()
    t[np.isnan(v)] = 0x7F
    return t, np.float32(1) / scale


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def norm_inputs(rows, cols, dt, rt, wt, seed):
    g = gen(seed)
    x = torch.randn(rows, cols, device="cuda", generator=g).to(dt)
    res = None if rt is None else (4 * torch.randn(rows, cols, device="cuda", generator=g)).to(rt)
    w = (1 + 0.3 * torch.randn(cols, device="cuda", generator=g)).to(wt)
    return x, res, w


def norm64(h, w, eps):
    h = h.double()
    rstd = 1 / (h.square().mean(1) + np.float32(eps)).sqrt()
    return rstd, h * rstd[:, None] * w.double()


def check_norm(r, x, res, w, eps, fmt, direction, want_y, pow2=False):
    h = x if res is None else (x.float() + res.float()).to(res.dtype)
    assert torch.equal(r["h"], h)
    rstd, y = norm64(h, w, eps)
    near(r["rstd"], rstd, rstd * 41 * U)
    assert (r["y"] is not None) == want_y and (r["q"] is not None) == bool(direction & 1) and (r["q_t"] is not None) == bool(direction & 2)
    if want_y:
        near(r["y"], y, y.abs() * (HALF[x.dtype] * (1 + 2.0 ** -7) + 43 * U) + 1e-40)
    if direction & 1:
        check_copy(r["q"], r["scale_inv"], y, fmt, 43 * U, pow2)
    if direction & 2:
        check_copy(r["q_t"], r["scale_inv_t"], y.t(), fmt, 43 * U, pow2)


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("rt", [None, BF16, FP32])
@pytest.mark.parametrize("rows,cols", [(16, 16), (144, 1040), (400, 7168)])
def test_norm_both_copies(dt, rt, rows, cols):
    fq = require_cuda()
    x, res, w = norm_inputs(rows, cols, dt, rt, FP32 if dt == BF16 else BF16, rows)
    r = fq.fp8q_rmsnorm(x, w, res, eps=1e-5, direction=fq.BOTH, want_y=True)
    check_norm(r, x, res, w, 1e-5, 0, 3, True)


@pytest.mark.parametrize("rows,cols", [(1, 7168), (3, 4096), (305, 272), (1000, 8192), (5, 16384), (700, 32768), (2, 128)])
def test_norm_row_copy(rows, cols):
    fq = require_cuda()
    x, res, w = norm_inputs(rows, cols, BF16, FP32 if rows % 2 else BF16, FP32, cols)
    r = fq.fp8q_rmsnorm(x, w, res, direction=fq.ROW)
    check_norm(r, x, res, w, 1e-6, 0, 1, False)


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (7, 3), (33, 1001), (310, 4097), (2, 8193), (3, 32767), (9, 24)])
def test_norm_any_columns(dt, rows, cols):
    """No copy: any number of columns."""
    fq = require_cuda()
    x, res, w = norm_inputs(rows, cols, dt, BF16, FP32, rows)
    r = fq.fp8q_rmsnorm(x, w, res, direction=0, want_y=True)
    check_norm(r, x, res, w, 1e-6, 0, 0, True)


@pytest.mark.parametrize("fmt,pow2,direction", [(1, False, 3), (0, True, 3), (1, True, 2), (0, False, 2)])
def test_norm_formats(fmt, pow2, direction):
    fq = require_cuda()
    x, res, w = norm_inputs(272, 784, BF16, None, BF16, 5)
    r = fq.fp8q_rmsnorm(x, w, fmt=fmt, pow2_scales=pow2, direction=direction)
    check_norm(r, x, res, w, 1e-6, fmt, direction, False, pow2)


def test_norm_codes_are_the_quantizer_s():
    """FP32 throughout: y shows the values that the copies were made from, so every code and scale is known."""
    fq = require_cuda()
    x, _, w = norm_inputs(160, 1072, FP32, None, FP32, 6)
    x[5] = 0
    x[7, 300] = float("nan")
    x[9, 40] = float("inf")
    for fmt, pow2 in ((0, False), (1, True)):
        r = fq.fp8q_rmsnorm(x, w, fmt=fmt, pow2_scales=pow2, direction=fq.BOTH, want_y=True)
        assert torch.isnan(r["y"][7]).all() and torch.isnan(r["y"][9, 40]) and (r["y"][9, :40] == 0).all() and (r["y"][5] == 0).all()
        for name, v in (("", r["y"]), ("_t", r["y"].t().contiguous())):
            q, inv = codes_of(v, fmt, pow2)
            np.testing.assert_array_equal(r["q" + name].cpu().numpy(), q)
            np.testing.assert_array_equal(r["scale_inv" + name].cpu().numpy().view(np.uint32), inv.view(np.uint32))


def test_norm_unaligned_views_and_guards():
    """Odd places without a copy; nothing beside the outputs is written."""
    fq = require_cuda()
    base = torch.randn(1 + 33 * 64, device="cuda", generator=gen(8)).bfloat16()
    x, w = base[1:].view(33, 64), torch.rand(65, device="cuda", generator=gen(9))[1:]
    bufs = {"y": Guarded((33, 64), BF16), "h": Guarded((33, 64), FP32), "rstd": Guarded((33,), FP32)}
    res = torch.randn(33, 64, device="cuda", generator=gen(10))
    r = fq.fp8q_rmsnorm(x, w, res, direction=0, want_y=True, out={k: b.t for k, b in bufs.items()})
    check_norm(r, x, res, w, 1e-6, 0, 0, True)
    bufs |= {"q": Guarded((48, 272)), "scale_inv": Guarded((48, 3), FP32), "q_t": Guarded((272, 48)), "scale_inv_t": Guarded((272, 1), FP32)}
    x, res, w = norm_inputs(48, 272, BF16, None, FP32, 11)
    r = fq.fp8q_rmsnorm(x, w, direction=fq.BOTH, out={k: bufs[k].t for k in ("q", "scale_inv", "q_t", "scale_inv_t")})
    check_norm(r, x, res, w, 1e-6, 0, 3, False)
    for b in bufs.values():
        b.check()


def test_norm_in_place_and_empty():
    fq = require_cuda()
    x, res, w = norm_inputs(64, 512, BF16, BF16, FP32, 12)
    keep = res.clone()
    r = fq.fp8q_rmsnorm(x, w, res, direction=fq.BOTH, want_y=True, out={"h": res})
    assert r["h"] is res
    check_norm(r, x, keep, w, 1e-6, 0, 3, True)
    e = fq.fp8q_rmsnorm(x[:0], w, res[:0], direction=fq.BOTH, want_y=True)
    assert e["q"].shape == (0, 512) and e["q_t"].shape == (512, 0)
    back = fq.fp8q_rmsnorm_backward(x[:0], res[:0], w, e["rstd"])
    assert back["d_x"].shape == (0, 512) and (back["d_weight"] == 0).all()


def check_norm_backward(got, d_y, h, w, rstd, d_h):
    rows, cols = h.shape
    d, hh, ww, r = d_y.double(), h.double(), w.double(), rstd.double()[:, None]
    g, u = d * ww, hh * r
    mean = (g * u).mean(1, keepdim=True)
    mags = (g * u).abs().mean(1, keepdim=True)
    d_x = r * (g - u * mean)
    tol = r * ((SUM + 6) * U * u.abs() * mags + 4 * U * (g.abs() + (u * mean).abs()))
    if d_h is not None:
        d_x = d_x + d_h.double()
    near(got["d_x"], d_x, tol + HALF[h.dtype] * (d_x.abs() + tol) * (1 + 2.0 ** -7) + 1e-40)
    near(got["d_weight"], (d * u).sum(0), (rows + 100) * U * (d * u).abs().sum(0))


@pytest.mark.parametrize("dt,ht,wt", [(BF16, BF16, FP32), (BF16, FP32, BF16), (FP32, BF16, FP32), (FP32, FP32, FP32)])
@pytest.mark.parametrize("rows,cols", [(1, 7168), (37, 16), (700, 4096), (2, 8200), (9, 32768), (5, 4097), (640, 33), (1, 1)])
def test_norm_backward(dt, ht, wt, rows, cols):
    fq = require_cuda()
    g = gen(rows + cols)
    h = (3 * torch.randn(rows, cols, device="cuda", generator=g)).to(ht)
    d_y = torch.randn(rows, cols, device="cuda", generator=g).to(dt)
    w = (1 + 0.3 * torch.randn(cols, device="cuda", generator=g)).to(wt)
    rstd = 1 / (h.float().square().mean(1) + 1e-6).sqrt()
    d_h = None if rows % 2 else torch.randn(rows, cols, device="cuda", generator=g).to(ht)
    out = {"d_x": Guarded((rows, cols), ht), "d_weight": Guarded((cols,), FP32)}
    got = fq.fp8q_rmsnorm_backward(d_y, h, w, rstd, d_h, out={k: b.t for k, b in out.items()})
    check_norm_backward(got, d_y, h, w, rstd, d_h)
    for b in out.values():
        b.check()
    if d_h is not None:  # in place
        want = got["d_x"].clone()
        assert torch.equal(fq.fp8q_rmsnorm_backward(d_y, h, w, rstd, d_h, out={"d_x": d_h})["d_x"], want)


# rows enough for CTAs that stay; columns whose rows start at every place of eight, the widest that stay and beyond
ODD = [(2500, 1), (2501, 7), (1219, 250), (3001, 1023), (700, 4097), (650, 4100), (333, 8185), (340, 8186)]


@pytest.mark.parametrize("dt,rt", [(BF16, None), (BF16, BF16), (FP32, FP32), (BF16, FP32), (FP32, None), (FP32, BF16)])
@pytest.mark.parametrize("rows,cols", ODD)
def test_norm_many_rows_of_any_columns(dt, rt, rows, cols):
    """A row's neighbours in its first and last eight values do not reach it, and are not written."""
    fq = require_cuda()
    x, res, w = norm_inputs(rows, cols, dt, rt, FP32 if cols % 2 else BF16, cols)
    x[17] = float("nan")
    x[rows - 2] = float("inf")
    bufs = {"y": Guarded((rows, cols), dt), "rstd": Guarded((rows,), FP32)} | ({"h": Guarded((rows, cols), rt)} if rt else {})
    r = fq.fp8q_rmsnorm(x, w, res, direction=0, want_y=True, out={k: b.t for k, b in bufs.items()})
    assert torch.isnan(r["y"][17]).all() and torch.isnan(r["y"]).sum(1).count_nonzero() == 2 and torch.isnan(r["rstd"]).sum() == 1
    keep = torch.tensor([i for i in range(rows) if i not in (17, rows - 2)], device="cuda")
    check_norm({k: r[k][keep] if k in ("h", "rstd", "y") else None for k in r}, x[keep], None if rt is None else res[keep], w, 1e-6, 0, 0, True)
    for b in bufs.values():
        b.check()
    if rt:  # in place, and the same values
        again = fq.fp8q_rmsnorm(x, w, res, direction=0, want_y=True, out={"h": res})
        for k in ("h", "rstd", "y"):
            assert torch.equal(again[k].nan_to_num(7.0), r[k].nan_to_num(7.0))


@pytest.mark.parametrize("dt,ht", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32)])
@pytest.mark.parametrize("rows,cols", ODD)
def test_norm_backward_many_rows_of_any_columns(dt, ht, rows, cols):
    fq = require_cuda()
    g = gen(rows + cols)
    h = (3 * torch.randn(rows, cols, device="cuda", generator=g)).to(ht)
    d_y = torch.randn(rows, cols, device="cuda", generator=g).to(dt)
    w = (1 + 0.3 * torch.randn(cols, device="cuda", generator=g)).to(ht)
    rstd = 1 / (h.float().square().mean(1) + 1e-6).sqrt()
    d_h = None if rows % 2 else torch.randn(rows, cols, device="cuda", generator=g).to(ht)
    out = {"d_x": Guarded((rows, cols), ht), "d_weight": Guarded((cols,), FP32)}
    got = fq.fp8q_rmsnorm_backward(d_y, h, w, rstd, d_h, out={k: b.t for k, b in out.items()})
    check_norm_backward(got, d_y, h, w, rstd, d_h)
    for b in out.values():
        b.check()
    d_y[21] = float("nan")  # stays in its row
    poisoned = fq.fp8q_rmsnorm_backward(d_y, h, w, rstd, d_h, out=None if d_h is None else {"d_x": d_h})
    keep = torch.arange(rows, device="cuda") != 21
    assert torch.equal(poisoned["d_x"][keep], got["d_x"][keep]) and torch.isnan(poisoned["d_x"][21]).all()
    assert torch.isnan(poisoned["d_weight"]).all()


def test_norm_gradient_against_differences():
    """A step of 2^-12 both ways in 64 bits: its error is some 2^-24 of the third derivative, far below the bound
    of 2^-14 of the sum of magnitudes, which also covers FP32."""
    fq = require_cuda()
    g = gen(3)
    x = torch.randn(24, 200, device="cuda", generator=g)
    w, d_y, vx, vw = (torch.randn(*s, device="cuda", generator=g) for s in ((200,), (24, 200), (24, 200), (200,)))
    r = fq.fp8q_rmsnorm(x, w, direction=0, want_y=True)
    got = fq.fp8q_rmsnorm_backward(d_y, x, w, r["rstd"])

    def f(e, dx, dw):
        return float((norm64(x.double() + e * dx.double(), w.double() + e * dw.double(), 1e-6)[1] * d_y.double()).sum())

    e = 2.0 ** -12
    for dx, dw, grad, v in ((vx, 0 * vw, got["d_x"], vx), (0 * vx, vw, got["d_weight"], vw)):
        diff = (f(e, dx, dw) - f(-e, dx, dw)) / (2 * e)
        each = grad.double() * v.double()
        assert abs(diff - float(each.sum())) <= 2.0 ** -14 * float(each.abs().sum())


# ---------------------------------------------------------------------------
# gated activation
# ---------------------------------------------------------------------------
# Of exp(-gate): 2 units of the exponential (4 u) and two roundings; 1 + e and its reciprocal (one unit): 3 u;
# three products.  The gradient's 1 - s takes two roundings more, and 1 + gate (1 - s) another.
# A sigmoid below 2^-126 counts as 0: a value is off by its other factors times 2^-126, TINY, at most.
REL, REL_GRAD, TINY = 16 * U, 24 * U, 2.0 ** -126


def gate64(h):
    gate, up = h.double().chunk(2, 1)
    return gate * torch.sigmoid(gate) * up


def gate_inputs(rows, inner, dt, seed):
    h = 2 * torch.randn(rows, 2 * inner, device="cuda", generator=gen(seed))
    h[0, :min(8, inner)] = torch.tensor([-90.0, -20.0, 0.0, -0.0, 20.0, 90.0, 1e-30, -1.2784645], device="cuda")[:min(8, inner)]
    return h.to(dt)


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("rows,inner,direction", [(16, 16, 3), (144, 1040, 3), (272, 2048, 2), (1, 2048, 1), (331, 144, 1), (5, 3, 0), (40, 1001, 0), (1, 1, 0)])
def test_gate(dt, rows, inner, direction):
    fq = require_cuda()
    h = gate_inputs(rows, inner, dt, rows)
    for fmt, pow2, want_a in ((0, False, direction == 0), (1, True, True)):
        r = fq.fp8q_swiglu(h, fmt=fmt, direction=direction, pow2_scales=pow2, want_a=want_a)
        a = gate64(h)
        assert (r["a"] is not None) == want_a and (r["q"] is not None) == bool(direction & 1) and (r["q_t"] is not None) == bool(direction & 2)
        if want_a:
            near(r["a"], a, a.abs() * (HALF[dt] * (1 + 2.0 ** -7) + REL) + 1e-38 + TINY * (h[:, :inner].double() * h[:, inner:].double()).abs())
        if direction & 1:
            check_copy(r["q"], r["scale_inv"], a, fmt, REL, pow2)
        if direction & 2:
            check_copy(r["q_t"], r["scale_inv_t"], a.t(), fmt, REL, pow2)


def gate_grad64(h, d_a):
    gate, up = h.double().chunk(2, 1)
    d, s, t = d_a.double(), torch.sigmoid(gate), torch.sigmoid(-gate)
    d_g, d_u = d * up * s * (1 + gate * t), d * gate * s
    # 1 + gate (1 - s) has a root near -1.28: its error is of its terms
    mags = torch.cat([(d * up * s).abs() * (1 + (gate * t).abs()), d_u.abs()], 1)
    flushed = torch.cat([(d * up).abs() * (1 + gate.abs()), (d * gate).abs()], 1) * (s < 2 * TINY).repeat(1, 2) * TINY
    return torch.cat([d_g, d_u], 1), mags + flushed / REL_GRAD


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("rows,inner,direction", [(16, 16, 3), (144, 1040, 3), (128, 136, 3), (272, 2048, 2), (1, 2048, 1), (331, 72, 1), (5, 3, 0), (40, 1001, 0)])
def test_gate_backward(dt, rows, inner, direction):
    """Inner sizes that are no multiple of 128 put both branches into one group."""
    fq = require_cuda()
    h = gate_inputs(rows, inner, dt, rows)
    d_a = torch.randn(rows, inner, device="cuda", generator=gen(1)).to(dt)
    want, mags = gate_grad64(h, d_a)
    r = fq.fp8q_swiglu_backward(h, d_a, direction=direction, want_d_h=True)
    near(r["d_h"], want, want.abs() * HALF[dt] * (1 + 2.0 ** -7) + REL_GRAD * mags + 1e-38)
    for name, w, m in (("q", want, mags), ("q_t", want.t(), mags.t())):
        if r[name] is None:
            continue
        inv = r["scale_inv" + name[1:]]
        wide = inv.double().repeat_interleave(128, 1)[:, :w.shape[1]]
        near(r[name].view(TYPES[1]).double() * wide, w, (w.abs() * CODE_HALF[1] + REL_GRAD * m) * (1 + 2 * REL_GRAD) + CODE_SUB[1] * wide + 8 * U * w.abs())


def test_gate_codes_are_the_quantizer_s():
    fq = require_cuda()
    h = gate_inputs(176, 592, FP32, 7)
    h[11, 100], h[12, 592 + 5], h[13] = float("nan"), float("inf"), 0.0
    h[14, 7] = torch.tensor(-1, dtype=torch.int32, device="cuda").view(FP32)  # a negative NaN
    h[15, 9], h[15, 10], h[15, 11] = float("-inf"), 1e38, -1e38
    h[20], h[21, :592], h[22, 592:] = h[20] * 1e-20, 1e-22, 3e-38  # groups whose scale is the largest FP32 number
    d_a = torch.randn(176, 592, device="cuda", generator=gen(2))
    r = fq.fp8q_swiglu(h, fmt=0, direction=fq.BOTH, want_a=True)
    b = fq.fp8q_swiglu_backward(h, d_a, fmt=1, direction=fq.BOTH, want_d_h=True)
    row = fq.fp8q_swiglu_backward(h, d_a, fmt=1, direction=fq.ROW)
    assert torch.equal(row["q"], b["q"]) and torch.equal(row["scale_inv"], b["scale_inv"])
    assert torch.equal(torch.isnan(r["a"]), torch.isnan(gate64(h))) and torch.equal(torch.isnan(b["d_h"]), torch.isnan(gate_grad64(h, d_a)[0]))
    for out, dense, fmt in ((r, r["a"], 0), (b, b["d_h"], 1)):
        for name, v in (("", dense), ("_t", dense.t().contiguous())):
            q, inv = codes_of(v, fmt)
            np.testing.assert_array_equal(out["q" + name].cpu().numpy(), q)
            np.testing.assert_array_equal(out["scale_inv" + name].cpu().numpy().view(np.uint32), inv.view(np.uint32))


def test_gate_gradient_against_differences():
    """As for the norm: steps of 2^-12 in 64 bits, bound 2^-14 of the sum of magnitudes."""
    fq = require_cuda()
    g = gen(4)
    h, v = (torch.randn(16, 240, device="cuda", generator=g) for _ in range(2))
    d_a = torch.randn(16, 120, device="cuda", generator=g)
    got = fq.fp8q_swiglu_backward(h, d_a, direction=0, want_d_h=True)["d_h"]
    e = 2.0 ** -12
    f = lambda s: float((gate64(h.double() + s * v.double()) * d_a.double()).sum())  # noqa: E731
    each = got.double() * v.double()
    assert abs((f(e) - f(-e)) / (2 * e) - float(each.sum())) <= 2.0 ** -14 * float(each.abs().sum())


def test_guards_of_the_copies():
    fq = require_cuda()
    h = gate_inputs(48, 200 // 8 * 8, BF16, 3)[:, :400].contiguous()
    d_a = torch.randn(48, 200, device="cuda", generator=gen(5)).bfloat16()
    bufs = {"q": Guarded((48, 400)), "scale_inv": Guarded((48, 4), FP32), "q_t": Guarded((400, 48)), "scale_inv_t": Guarded((400, 1), FP32),
            "d_h": Guarded((48, 400), BF16)}
    fq.fp8q_swiglu_backward(h, d_a, want_d_h=True, out={k: b.t for k, b in bufs.items()})
    for b in bufs.values():
        b.check()


# ---------------------------------------------------------------------------
# past 32 bits
# ---------------------------------------------------------------------------
def test_offsets_past_32_bits():
    """More than 2^31 values: the last rows (the last 128 of the transposed copies' groups) are those of a call on them alone."""
    fq = require_cuda()
    rows, cols, tail = 135168, 16384, 256
    h = torch.empty(rows, cols, dtype=BF16, device="cuda").normal_(generator=gen(50))
    assert h.numel() > 2 ** 31
    w = torch.rand(cols, device="cuda", generator=gen(51))
    last = h[-tail:].contiguous()
    big, small = fq.fp8q_swiglu(h, direction=fq.BOTH), fq.fp8q_swiglu(last, direction=fq.BOTH)
    for name in ("q", "scale_inv"):
        assert torch.equal(big[name][-tail:], small[name])
    assert torch.equal(big["q_t"][:, -tail:], small["q_t"]) and torch.equal(big["scale_inv_t"][:, -tail // 128:], small["scale_inv_t"])
    d_a = torch.empty(rows, cols // 2, dtype=BF16, device="cuda").normal_(generator=gen(52))
    big, small = fq.fp8q_swiglu_backward(h, d_a), fq.fp8q_swiglu_backward(last, d_a[-tail:].contiguous())
    assert torch.equal(big["q"][-tail:], small["q"]) and torch.equal(big["q_t"][:, -tail:], small["q_t"])
    del big, d_a
    big, small = fq.fp8q_rmsnorm(h, w, h, direction=fq.BOTH), fq.fp8q_rmsnorm(last, w, last, direction=fq.BOTH)
    assert torch.equal(big["h"][-tail:], small["h"]) and torch.equal(big["q"][-tail:], small["q"])
    assert torch.equal(big["q_t"][:, -tail:], small["q_t"])
    d, e = fq.fp8q_rmsnorm_backward(h, big["h"], w, big["rstd"]), fq.fp8q_rmsnorm_backward(last, small["h"], w, small["rstd"])
    assert torch.equal(d["d_x"][-tail:], e["d_x"])


# ---------------------------------------------------------------------------
# streams, graphs, refusals
# ---------------------------------------------------------------------------
def test_streams_and_graphs():
    """The same bits on a side stream and from a replayed graph with new inputs."""
    fq = require_cuda()
    x, res, w = norm_inputs(256, 1024, BF16, BF16, FP32, 20)
    d_y = torch.randn(256, 1024, device="cuda", generator=gen(21)).bfloat16()

    def step():
        r = fq.fp8q_rmsnorm(x, w, res, direction=fq.BOTH, want_y=True)
        b = fq.fp8q_rmsnorm_backward(d_y, r["h"], w, r["rstd"], d_h=res)
        s = fq.fp8q_swiglu(r["y"], direction=fq.BOTH)
        t = fq.fp8q_swiglu_backward(r["y"], d_y[:, :512].contiguous())
        return [v for d in (r, b, s, t) for v in d.values() if v is not None]

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(2):
        x.copy_(torch.randn(256, 1024, device="cuda", generator=gen(30 + i)))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_refusals():
    fq = require_cuda()
    x, res, w = norm_inputs(16, 64, BF16, BF16, FP32, 40)
    ok = fq.fp8q_rmsnorm(x, w, res)
    for call in (lambda: fq.fp8q_rmsnorm(x.half(), w), lambda: fq.fp8q_rmsnorm(x, w[:63]), lambda: fq.fp8q_rmsnorm(x, w, res[:8]),
                 lambda: fq.fp8q_rmsnorm(x[:, :32], w[:32]), lambda: fq.fp8q_rmsnorm(x.cpu(), w), lambda: fq.fp8q_rmsnorm(x, w.cpu()),
                 lambda: fq.fp8q_rmsnorm(x, w, out={"q": torch.empty(16, 32, dtype=torch.uint8, device="cuda")}),
                 lambda: fq.fp8q_rmsnorm_backward(x, res.float(), w, ok["rstd"], d_h=res), lambda: fq.fp8q_rmsnorm_backward(x, res, w, ok["rstd"][:3]),
                 lambda: fq.fp8q_swiglu(x[:, :63].contiguous()), lambda: fq.fp8q_swiglu_backward(x, x), lambda: fq.fp8q_swiglu_backward(x, x[:, :32].float())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fq.fp8q_rmsnorm(x[:, :24].contiguous(), w[:24]), lambda: fq.fp8q_rmsnorm(x[:9], w, direction=fq.COL),
                 lambda: fq.fp8q_rmsnorm(x, w, eps=-1.0), lambda: fq.fp8q_rmsnorm(x, w, direction=7), lambda: fq.fp8q_swiglu(x, direction=0),
                 lambda: fq.fp8q_swiglu(x, fmt=2)):
        with pytest.raises(fq.Fp8qError):
            call()
