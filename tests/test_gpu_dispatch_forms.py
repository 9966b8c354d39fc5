"""Dispatch and rowwise quantizer: alignments, types and scale rules that the sizes of test_gpu_moe.py do not
reach, bit for bit against the oracle."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import Guarded, host, require_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("direction", ["COL", "BOTH"])
def test_transposed_codes_that_start_between_32_byte_lines(fmt, direction):
    """Columns of a multiple of 32 rows whose buffer starts 16 bytes off a line take the 16-byte stores."""
    fq = require_cuda()
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn(70, 272, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, 5, (70, 3), generator=g, device="cuda").int()
    p = fq.fp8q_moe_plan(ids, 5, 32)
    rows = p["src"].numel()
    assert rows % 32 == 0
    raw = torch.full((272 * rows + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    q_t = raw[16:16 + 272 * rows].view(272, rows)
    assert q_t.data_ptr() % 32 == 16
    r = fq.fp8q_moe_dispatch(x, p, fmt, getattr(fq, direction), out={"q_t": q_t})
    src = p["src"].long()
    xg = torch.where((src >= 0)[:, None], x[src.clamp_min(0) // 3], torch.zeros_like(x[:1]))
    q, si = oracle.blockwise(host(xg.view(torch.int16)).view(np.uint16), fmt, (128, 1), False)
    np.testing.assert_array_equal(host(q_t), q.T)
    np.testing.assert_array_equal(host(r["scale_inv_t"]).view(np.uint32), np.ascontiguousarray(si.T).view(np.uint32))
    assert (raw[:16] == 0xA5).all() and (raw[16 + 272 * rows:] == 0xA5).all()


@pytest.mark.parametrize("rows", [1, 17, 129])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("pow2", [False, True])
def test_rowwise_quantizer_of_any_rows_in_every_form(rows, fmt, pow2):
    fq = require_cuda()
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn(rows, 400, device="cuda", generator=g) * torch.exp2(9 * torch.randn(rows, 1, device="cuda", generator=g))).bfloat16()
    x[rows // 2, 5] = 0.0
    x[rows // 2, 300] = float("inf")
    for block in (fq.BLOCK_1X128, fq.BLOCK_128X128):
        out = {"q": Guarded((rows, 400)), "scale_inv": Guarded((rows if block == 1 else -(-rows // 128), 4), torch.float32)}
        r = fq.fp8q_quantize_blockwise(x, fmt, block, pow2_scales=pow2, out={k: v.t for k, v in out.items()})
        q, si = oracle.blockwise(host(x.view(torch.int16)).view(np.uint16), fmt, (1, 128) if block == 1 else (128, 128), pow2)
        np.testing.assert_array_equal(host(r["q"]), q)
        np.testing.assert_array_equal(host(r["scale_inv"]).view(np.uint32), si.view(np.uint32))
        for b in out.values():
            b.check()
