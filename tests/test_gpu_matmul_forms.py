"""Products of blockwise FP8 tensors: forms, tiles and limits that the sizes of test_gpu_matmul.py do not reach.
Its tolerance holds here, too: (128 + KB + 4) * 2^-23 of the sum of the terms' magnitudes and half a unit of
the output type."""
import time

import pytest
import torch

from gpu_util import Guarded, require_cuda
from test_gpu_matmul import check, codes, gen, scales, values

pytestmark = pytest.mark.gpu


FORMS = [(1, 512, 4096, 128), (100, 2048, 2048, 1), (130, 256, 4096, 128), (600, 4096, 2048, 1), (40, 40000, 400, 1)]


@pytest.mark.parametrize("m,n,k,block", FORMS)
@pytest.mark.parametrize("budget_ns", [1, 1000, 100_000])
def test_a_short_wait_budget_does_not_end_a_healthy_product(m, n, k, block, budget_ns):
    """A wait may give up once the budget is over and some 100 us have passed; a healthy product's waits last a
    few microseconds, so it ends as ever however short the budget."""
    fq = require_cuda()
    g = gen(m + n)
    kb = k // 128 + (k % 128 > 0)
    a, b = codes(g, (m, k), 0), codes(g, (n, k), 0)
    sa, sb = scales(g, (m, kb)), scales(g, (-(-n // block), kb))
    want = fq.fp8q_matmul_blockwise(a, sa, b, sb, b_block=block, out_dtype=torch.float32)
    fq.check_device()
    try:
        fq.set_wait_budget_ns(budget_ns)
        for _ in range(5):
            got = fq.fp8q_matmul_blockwise(a, sa, b, sb, b_block=block, out_dtype=torch.float32)
            fq.check_device()
            assert torch.equal(got, want)
    finally:
        fq.set_wait_budget_ns(1_000_000_000)


@pytest.mark.parametrize("m,n,k,block", [f for f in FORMS if f[1] != 40000])
def test_a_wait_lasts_as_long_as_its_budget(m, n, k, block):
    """Without loads the call takes the budget (no wait gives up before) and not several of them: the waits of
    one call run side by side, and an expired one ends the others of its CTA."""
    fq = require_cuda()
    g = gen(m + n)
    kb = k // 128
    a, b = codes(g, (m, k), 0), codes(g, (n, k), 0)
    sa, sb = scales(g, (m, kb)), scales(g, (-(-n // block), kb))
    fq.fp8q_matmul_blockwise(a, sa, b, sb, b_block=block)
    fq.check_device()
    budget = 0.2
    try:
        fq.set_wait_budget_ns(int(budget * 1e9))
        fq.debug_stall_matmul_loads(True)
        torch.cuda.synchronize()
        start = time.perf_counter()
        fq.fp8q_matmul_blockwise(a, sa, b, sb, b_block=block)
        torch.cuda.synchronize()
        took = time.perf_counter() - start
        with pytest.raises(fq.Fp8qError, match="gave up"):
            fq.check_device()
    finally:
        fq.debug_stall_matmul_loads(False)
        fq.set_wait_budget_ns(1_000_000_000)
    assert budget <= took < 5 * budget


@pytest.mark.parametrize("rows", [40, 400])
def test_a_short_wait_budget_does_not_end_a_product_that_waits_for_memory(rows):
    """Weights of 40 experts, 168 MB, come from HBM: a warp of sums waits for microseconds."""
    fq = require_cuda()
    g = gen(rows)
    b, sb = codes(g, (40, 2048, 2048), 0), scales(g, (40, 16, 16))
    a, sa = codes(g, (rows, 2048), 0), scales(g, (rows, 16))
    off = [rows * i // 40 for i in range(41)]
    flush = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    want = fq.fp8q_matmul_grouped(a, sa, b, sb, off, out_dtype=torch.float32)
    fq.check_device()
    try:
        fq.set_wait_budget_ns(1)
        for _ in range(5):
            flush.zero_()
            got = fq.fp8q_matmul_grouped(a, sa, b, sb, off, out_dtype=torch.float32)
            fq.check_device()
            assert torch.equal(got, want)
    finally:
        fq.set_wait_budget_ns(1_000_000_000)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offsets", [[0, 4, 9], [3, 3, 8], [2, 2, 2], [-4, 5, 100]])
@pytest.mark.parametrize("n", [48, 37])
def test_empty_reduction_of_groups_leaves_the_other_rows_alone(out_dtype, offsets, n):
    """An empty sum is zero for the groups' rows, and rows in no group are not written."""
    fq = require_cuda()
    a, sa = torch.empty(12, 0, dtype=torch.uint8, device="cuda"), torch.empty(12, 0, device="cuda")
    b = torch.empty(2, n, 0, dtype=torch.uint8, device="cuda")
    sb = torch.empty(2, 1, 0, device="cuda")
    out = Guarded((12, n), out_dtype)
    out.t.fill_(7.0)
    fq.fp8q_matmul_grouped(a, sa, b, sb, offsets, out_dtype=out_dtype, out=out.t)
    fq.check_device()
    out.check()
    lo, hi = max(offsets[0], 0), min(offsets[-1], 12)
    want = torch.full_like(out.t, 7.0)
    want[lo:hi] = 0.0
    assert torch.equal(out.t, want)


@pytest.mark.parametrize("m,n,k", [(2700, 2820, 400), (100, 40000, 400), (2700, 2820, 128)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_column_scales_over_several_tiles(m, n, k, out_dtype):
    """More tiles than pairs (11 x 12) or CTAs (157), with reductions that are no multiple of the scales' four
    blocks or the two of tensor memory: the rings go on from one tile to the next."""
    fq = require_cuda()
    g = gen(m + k)
    kb = -(-k // 128)
    a, b = codes(g, (m, k), 1), codes(g, (n, k), 0)
    sa, sb = scales(g, (m, kb)), scales(g, (n, kb))
    out = Guarded((m, n), out_dtype)
    fq.fp8q_matmul_blockwise(a, sa, b, sb, 1, 0, 1, out_dtype, out=out.t)
    fq.check_device()
    out.check()
    check(out.t, values(a, sa, 1, 1), values(b, sb, 0, 1))


@pytest.mark.parametrize("accumulate", [False, True])
def test_grouped_wgrad_over_several_tiles(accumulate):
    """9 experts of 4 x 5 tiles over 76 pairs, with 0 to 11 blocks of rows each."""
    fq = require_cuda()
    g = gen(21)
    m, n = 1000, 1230
    blocks = [3, 0, 1, 11, 2, 5, 0, 7, 4]
    off = [0]
    for c in blocks:
        off.append(off[-1] + 128 * c)
    rows = off[-1]
    a, b = codes(g, (m, rows), 1), codes(g, (n, rows), 0)
    sa, sb = scales(g, (m, rows // 128)), scales(g, (n, rows // 128))
    out = Guarded((len(blocks), m, n), torch.float32)
    start = torch.randn(len(blocks), m, n, device="cuda", generator=g)
    out.t.copy_(start)
    fq.fp8q_matmul_grouped_wgrad(a, sa, b, sb, off, 1, 0, accumulate=accumulate, out=out.t)
    fq.check_device()
    out.check()
    av, bv = values(a, sa, 1, 1), values(b, sb, 0, 1)
    for i in range(len(blocks)):
        lo, hi = off[i], off[i + 1]
        check(out.t[i], av[:, lo:hi], bv[:, lo:hi], start[i].double() if accumulate else None)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("a_fmt", [0, 1])
def test_grouped_pairs_over_several_tiles(out_dtype, a_fmt):
    """Groups of more than 128 rows on average take pairs: 14 row tiles of 12 column tiles over 76 pairs, from
    any row, with groups that are empty or end inside a tile."""
    fq = require_cuda()
    g = gen(22)
    off, n, k = [5, 5, 700, 701, 1500, 1756, 3000], 3000, 656
    rows = off[-1] + 20
    a, b = codes(g, (rows, k), a_fmt), codes(g, (6, n, k), 0)
    sa, sb = scales(g, (rows, 6)), scales(g, (6, 24, 6))
    out = Guarded((rows, n), out_dtype)
    out.t.fill_(7.0)
    fq.fp8q_matmul_grouped(a, sa, b, sb, off, a_fmt, 0, out_dtype, out=out.t)
    fq.check_device()
    out.check()
    av = values(a, sa, a_fmt, 1)
    for i in range(6):
        lo, hi = off[i], off[i + 1]
        if hi > lo:
            check(out.t[lo:hi], av[lo:hi], values(b[i], sb[i], 0, 128))
    assert (out.t[:5] == 7.0).all() and (out.t[3000:] == 7.0).all()
