"""The norm without a residual where CTAs stay: rows side by side in a CTA, chunks of columns behind the row, a last
set of rows that is not full, and the widest rows; the transposed copy with several tiles a CTA; and the copies in
the products that they are made for.  The bounds are those of test_gpu_norm_gate.py."""
import numpy as np
import pytest
import torch

from gpu_util import Guarded, require_cuda
from test_gpu_norm_gate import BF16, FP32, check_norm, codes_of, norm_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("rows,cols", [(5003, 272), (2501, 1040), (1000, 2064), (1219, 4112), (777, 8208), (700, 16384), (701, 11216), (9001, 16)])
def test_rows_without_a_residual(dt, rows, cols):
    """Rows of NaN at both ends and one with Inf reach no other row."""
    fq = require_cuda()
    assert rows > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    x, _, w = norm_inputs(rows, cols, dt, None, FP32 if dt == BF16 else BF16, cols)
    x[0], x[rows - 1], x[rows // 2, cols - 1] = float("nan"), float("nan"), float("inf")
    buf = {"y": Guarded((rows, cols), dt), "rstd": Guarded((rows,), FP32), "q": Guarded((rows, cols)), "scale_inv": Guarded((rows, -(-cols // 128)), FP32)}
    r = fq.fp8q_rmsnorm(x, w, direction=fq.ROW, want_y=True, out={k: b.t for k, b in buf.items()})
    for b in buf.values():
        b.check()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[[0, rows // 2, rows - 1]] = False
    assert torch.isnan(r["y"][0]).all() and torch.isnan(r["y"][rows - 1]).all() and torch.isnan(r["y"]).any(1).sum() == 3
    kept = {k: None if v is None else v[keep] for k, v in r.items()}
    check_norm(kept, x[keep], None, w, 1e-6, 0, 1, True)
    if dt == FP32:
        q, inv = codes_of(kept["y"], 0)
        np.testing.assert_array_equal(kept["q"].cpu().numpy(), q)
        np.testing.assert_array_equal(kept["scale_inv"].cpu().numpy().view(np.uint32), inv.view(np.uint32))
    alone = fq.fp8q_rmsnorm(x, w, direction=fq.ROW)
    assert torch.equal(alone["q"], r["q"]) and torch.equal(alone["scale_inv"], r["scale_inv"])
    dense = fq.fp8q_rmsnorm(x, w, direction=0, want_y=True)
    assert torch.equal(dense["y"][keep], kept["y"]) and torch.equal(dense["rstd"][keep], kept["rstd"])


@pytest.mark.parametrize("dt,rt", [(BF16, BF16), (FP32, None), (BF16, FP32)])
@pytest.mark.parametrize("rows,cols", [(4112, 4096), (6160, 2064)])
def test_several_transposed_tiles_a_cta(dt, rt, rows, cols):
    fq = require_cuda()
    assert -(-rows // 128) * -(-cols // 128) >= 3 * torch.cuda.get_device_properties(0).multi_processor_count
    x, res, w = norm_inputs(rows, cols, dt, rt, FP32, rows)
    buf = {"q_t": Guarded((cols, rows)), "scale_inv_t": Guarded((cols, -(-rows // 128)), FP32)}
    r = fq.fp8q_rmsnorm(x, w, res, direction=fq.BOTH, want_y=True, out={k: b.t for k, b in buf.items()})
    for b in buf.values():
        b.check()
    check_norm(r, x, res, w, 1e-6, 0, 3, True)
    if dt == FP32:
        q, inv = codes_of(r["y"].t().contiguous(), 0)
        np.testing.assert_array_equal(r["q_t"].cpu().numpy(), q)
        np.testing.assert_array_equal(r["scale_inv_t"].cpu().numpy().view(np.uint32), inv.view(np.uint32))


def test_a_linear_layer_on_the_copies():
    """y W^T of the row copy and d_out^T y of the transposed one, against FP32: a product of values rounded to E4M3 is
    off by sqrt(2^-8 + 2^-8) in the norm at most, one with an E5M2 factor by sqrt(2^-6 + 2^-8), and its BF16 by 2^-8."""
    fq = require_cuda()
    tokens, cols, out = 384, 512, 640
    x, res, w = norm_inputs(tokens, cols, BF16, BF16, FP32, 3)
    weight, d_out = (torch.randn(*s, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).bfloat16() for s in ((out, cols), (tokens, out)))
    n = fq.fp8q_rmsnorm(x, w, res, direction=fq.BOTH, want_y=True)
    qw = fq.fp8q_quantize_blockwise(weight, fq.E4M3, block=fq.BLOCK_128X128)
    qd = fq.fp8q_quantize_blockwise(d_out, fq.E5M2, direction=fq.BOTH)
    y = n["y"].float()
    fprop = fq.fp8q_matmul_blockwise(n["q"], n["scale_inv"], qw["q"], qw["scale_inv"])
    wgrad = fq.fp8q_matmul_blockwise(qd["q_t"], qd["scale_inv_t"], n["q_t"], n["scale_inv_t"], a_fmt=fq.E5M2, b_block=fq.BLOCK_1X128)
    for got, want, off in ((fprop, y @ weight.float().t(), (2 ** -7) ** 0.5), (wgrad, d_out.float().t() @ y, (2 ** -6 + 2 ** -8) ** 0.5)):
        assert got.shape == want.shape and (got.float() - want).norm() < (off + 2 ** -7) * want.norm()


@pytest.mark.parametrize("dt,rt", [(BF16, BF16), (BF16, None), (FP32, FP32), (FP32, None)])
@pytest.mark.parametrize("rows,cols", [(1, 4097), (2, 4096), (1, 4104), (3, 4112), (304, 4112), (2, 5121), (5, 8185), (303, 8191), (7, 8192)])
def test_few_rows_on_both_sides_of_4096_columns(dt, rt, rows, cols):
    fq = require_cuda()
    x, res, w = norm_inputs(rows, cols, dt, rt, FP32, rows + cols)
    row = cols % 16 == 0
    buf = {"y": Guarded((rows, cols), dt), "rstd": Guarded((rows,), FP32)} | ({"h": Guarded((rows, cols), rt)} if rt else {})
    if row:
        buf |= {"q": Guarded((rows, cols)), "scale_inv": Guarded((rows, -(-cols // 128)), FP32)}
    r = fq.fp8q_rmsnorm(x, w, res, direction=fq.ROW if row else 0, want_y=True, out={k: b.t for k, b in buf.items()})
    for b in buf.values():
        b.check()
    check_norm(r, x, res, w, 1e-6, 0, int(row), True)
    if rt:  # in place
        again = fq.fp8q_rmsnorm(x, w, res, direction=fq.ROW if row else 0, want_y=True, out={"h": res})
        assert torch.equal(again["h"], r["h"]) and torch.equal(again["y"], r["y"])
