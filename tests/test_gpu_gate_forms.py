"""The gated activation, its gradient and their copies where CTAs stay and take several tiles: the row copy alone,
whose rows may end anywhere, and both copies, with halves that are whole tiles (one set of inputs for both) and
that are not.  The bounds are those of test_gpu_norm_gate.py; FP32 inputs show the values that the codes were
made from, so that every code and scale is known."""
import numpy as np
import pytest
import torch

from gpu_util import Guarded, require_cuda
from test_gpu_norm_gate import (BF16, CODE_HALF, CODE_SUB, FP32, HALF, REL, REL_GRAD, TINY, TYPES, U, check_copy, codes_of, gate64, gate_grad64,
                                gate_inputs, gen, near)

pytestmark = pytest.mark.gpu


def tiles(rows, cols):
    return -(-rows // 128) * -(-cols // 128)


def buffers(rows, cols, direction, dense, dt):
    b = {dense: Guarded((rows, cols), dt)}
    if direction & 1:
        b |= {"q": Guarded((rows, cols)), "scale_inv": Guarded((rows, -(-cols // 128)), FP32)}
    if direction & 2:
        b |= {"q_t": Guarded((cols, rows)), "scale_inv_t": Guarded((cols, -(-rows // 128)), FP32)}
    return b


def exact_codes(r, dense, fmt):
    for name, v in (("", dense), ("_t", dense.t().contiguous())):
        if r["q" + name] is None:
            continue
        q, inv = codes_of(v, fmt)
        np.testing.assert_array_equal(r["q" + name].cpu().numpy(), q)
        np.testing.assert_array_equal(r["scale_inv" + name].cpu().numpy().view(np.uint32), inv.view(np.uint32))


def without_dense(fn, r, buf, **kw):
    """The same copies where the dense output is not asked for."""
    other = fn(**kw)
    for k in ("q", "scale_inv", "q_t", "scale_inv_t"):
        assert (r[k] is None) == (other[k] is None) and (r[k] is None or torch.equal(r[k].view(torch.uint8), other[k].view(torch.uint8)))
    for b in buf.values():
        b.check()


# rows that end inside a tile and inside a thread's eight, groups that end inside a tile
FORWARD = [(4099, 2048, 1), (7301, 1040, 1), (12345, 656, 1), (4112, 2048, 3), (7312, 1040, 3), (7312, 1040, 2)]
BACKWARD = [(9731, 2048, 1), (31111, 640, 1), (4099, 1928, 1), (7301, 520, 1), (4112, 2048, 3), (6160, 1032, 3), (7312, 1024, 2)]


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("rows,inner,direction", FORWARD)
def test_tiles(dt, rows, inner, direction):
    fq = require_cuda()
    assert tiles(rows, inner) >= 3 * torch.cuda.get_device_properties(0).multi_processor_count
    h = gate_inputs(rows, inner, dt, rows)
    h[rows - 1], h[130, 3] = 0.0, float("nan")
    buf = buffers(rows, inner, direction, "a", dt)
    r = fq.fp8q_swiglu(h, direction=direction, want_a=True, out={k: b.t for k, b in buf.items()})
    without_dense(fq.fp8q_swiglu, r, buf, h=h, direction=direction)
    if dt == FP32:
        exact_codes(r, r["a"], 0)
    assert torch.isnan(r["a"][130, 3]) and torch.isnan(r["a"]).sum() == 1
    a = gate64(h).nan_to_num(0.0)
    near(r["a"].nan_to_num(0.0), a, a.abs() * (HALF[dt] * (1 + 2.0 ** -7) + REL) + 1e-38 + TINY * (h[:, :inner].double() * h[:, inner:].double()).nan_to_num(0.0).abs())
    keep = torch.arange(rows, device="cuda") != 130
    if direction & 1:
        check_copy(r["q"][keep], r["scale_inv"][keep], a[keep], 0, REL)
    if direction & 2:
        cols = torch.arange(inner, device="cuda") != 3
        check_copy(r["q_t"][cols], r["scale_inv_t"][cols], a.t()[cols], 0, REL)


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("rows,inner,direction", BACKWARD)
def test_gradient_tiles(dt, rows, inner, direction):
    fq = require_cuda()
    pairs = inner % 128 == 0
    assert tiles(rows, 2 * inner) // (2 if pairs else 1) >= (8 if pairs and direction == 1 else 3) * torch.cuda.get_device_properties(0).multi_processor_count
    h = gate_inputs(rows, inner, dt, rows)
    d_a = torch.randn(rows, inner, device="cuda", generator=gen(1)).to(dt)
    h[rows - 1] = 0.0
    buf = buffers(rows, 2 * inner, direction, "d_h", dt)
    r = fq.fp8q_swiglu_backward(h, d_a, direction=direction, want_d_h=True, out={k: b.t for k, b in buf.items()})
    without_dense(fq.fp8q_swiglu_backward, r, buf, h=h, d_a=d_a, direction=direction)
    if dt == FP32:
        exact_codes(r, r["d_h"], 1)
    want, mags = gate_grad64(h, d_a)
    near(r["d_h"], want, want.abs() * HALF[dt] * (1 + 2.0 ** -7) + REL_GRAD * mags + 1e-38)
    for name, w, m in (("q", want, mags), ("q_t", want.t(), mags.t())):
        if r[name] is not None:
            wide = r["scale_inv" + name[1:]].double().repeat_interleave(128, 1)[:, :w.shape[1]]
            near(r[name].view(TYPES[1]).double() * wide, w, (w.abs() * CODE_HALF[1] + REL_GRAD * m) * (1 + 2 * REL_GRAD) + CODE_SUB[1] * wide + 8 * U * w.abs())
