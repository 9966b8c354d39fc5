"""The gated activation and its gradient where products of two inputs leave FP32's range but the result does not.

With u = 2^-24, to the tolerances of test_gpu_norm_gate.py (16 u, 24 u for the gradient, of each term; a sigmoid
below 2^-126 counts as 0, of gates from some -90 on) comes the rounding of a subnormal product on the way, 2^-150
times the factor that is multiplied in last."""
import pytest
import torch

from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
REL, REL_GRAD, TINY, SUB = 16 * U, 24 * U, 2.0 ** -126, 2.0 ** -150
BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, FP32: U}
GATES = [-3e38, -1e38, -1e30, -200.0, -100.0, -88.0, -87.0, -60.0, -30.0, -5.0, -1.0, -1e-30, 0.0, 1e-30, 0.7, 2.4, 5.0, 100.0, 1e30, 1e38]
SIZES = [0.0, 1e-38, -1e-20, 1e-3, 0.5, -1.0, 3e3, -1e20, 1e30, -1e37, 1e38, 3e38]


def table(rows, inner, dt):
    """Every gate with every up and every d_a, in an order that puts all of them into many groups."""
    g, u, d = torch.meshgrid(*(torch.tensor(v, device="cuda").to(dt) for v in (GATES, SIZES, SIZES)), indexing="ij")
    n = g.numel()
    pick = (torch.arange(rows * inner, device="cuda") * 1009 % n).view(rows, inner)  # 1009 and n have no common factor
    assert rows * inner >= n and n % 1009
    g, u, d = (t.flatten()[pick] for t in (g, u, d))
    return torch.cat([g, u], 1).contiguous(), d.contiguous()


def near(got, want, tol, dt):
    """Within tol, or beyond the type's largest number where `want` is, or may be."""
    largest = torch.finfo(dt).max
    tol = tol + want.abs() * HALF[dt] * (1 + 2.0 ** -7) + (2.0 ** -134 if dt == BF16 else SUB)
    assert not torch.isnan(got).any(), int(torch.isnan(got).sum())
    over = torch.isinf(got)
    assert (want.abs() + tol)[over].ge(largest).all() and (want[over].sign() == got[over].sign()).all()
    near_top = (want.abs() + tol) >= largest
    bad = ((got.double() - want).abs() > tol) & ~over & ~near_top
    assert not bad.any(), (int(bad.sum()), got[bad][:5], want[bad][:5])


def forward64(h):
    gate, up = h.double().chunk(2, 1)
    s = torch.sigmoid(gate)
    a = gate * s * up
    return a, REL * a.abs() + (s < 2 * TINY) * TINY * gate.abs().clamp_max(91) * up.abs() + SUB * up.abs()


def backward64(h, d):
    gate, up = h.double().chunk(2, 1)
    d, s, t = d.double(), torch.sigmoid(gate), torch.sigmoid(-gate)
    flushed = (s < 2 * TINY) * TINY * (1 + gate.abs().clamp_max(91))
    d_g, d_u = s * (1 + gate * t) * up * d, gate * s * d
    tol_g = (REL_GRAD * s * (1 + (gate * t).abs()) + flushed) * (up * d).abs() + SUB * torch.minimum(up.abs(), d.abs())
    return torch.cat([d_g, d_u], 1), torch.cat([tol_g, REL_GRAD * d_u.abs() + flushed * d.abs() + SUB * d.abs()], 1)


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("rows,inner,direction", [(16, 256, 3), (48, 144, 3), (33, 256, 1), (27, 136, 1), (16, 256, 0), (41, 131, 0), (4099, 2048, 1)])
def test_products_beyond_fp32(dt, rows, inner, direction):
    fq = require_cuda()
    h, d = table(rows, inner, dt)
    if not direction or inner % 16 == 0:
        want, tol = forward64(h)
        near(fq.fp8q_swiglu(h, direction=direction, want_a=True)["a"], want, tol, dt)
    want, tol = backward64(h, d)
    near(fq.fp8q_swiglu_backward(h, d, direction=direction, want_d_h=True)["d_h"], want, tol, dt)


def test_the_group_of_a_large_negative_gate_keeps_its_scale():
    """silu of -1e38 is 0 whatever the up branch holds: the other values of its groups are coded as they are without it."""
    fq = require_cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(16, 256, device="cuda", generator=g)
    h[:, 5], h[:, 128 + 5] = -1e38, 1e4
    clean = h.clone()
    clean[:, 5] = 0.0
    a, b = fq.fp8q_swiglu(h, direction=fq.BOTH), fq.fp8q_swiglu(clean, direction=fq.BOTH)
    assert torch.equal(a["scale_inv"], b["scale_inv"]) and torch.equal(a["scale_inv_t"], b["scale_inv_t"])
    assert torch.equal(a["q"] & 0x7F, b["q"] & 0x7F) and torch.equal(a["q_t"] & 0x7F, b["q_t"] & 0x7F)
