"""Products of blockwise FP8 tensors against the sum in 64 bits.

Tolerance.  A block's 128 products are exact in FP32 and summed by the tensor
core in at least 23 bits; the sums over the KB blocks and the two scale
products are FP32.  Every element is therefore within (128 + KB + 4) * 2^-23
of the sum of the terms' magnitudes, plus half a unit of the output type."""
import numpy as np
import pytest
import torch

from gpu_util import Guarded, require_cuda

pytestmark = pytest.mark.gpu

FP8 = (torch.float8_e4m3fn, torch.float8_e5m2)


def codes(g, shape, fmt):
    """Random finite codes of every exponent (E4M3 NaN is 0x7F, E5M2's top exponent is not finite)."""
    q = torch.randint(0, 256, shape, generator=g, device="cuda").to(torch.uint8)
    top = 0x7F if fmt == 0 else 0x7C
    return torch.where((q & 0x7F) >= top, q & 0x83, q)


def scales(g, shape):
    return torch.exp2(torch.empty(shape, device="cuda").uniform_(-6, 2, generator=g))


def values(q, s, fmt, rows_per_scale):
    """The tensor the codes stand for, in 64 bits."""
    v = q.view(FP8[fmt]).double()
    r = torch.arange(q.shape[-2], device="cuda") // rows_per_scale
    c = torch.arange(q.shape[-1], device="cuda") // 128
    return v * s.double()[..., r, :][..., c]


def check(got, a, b, extra=None):
    want, size = a @ b.T, a.abs() @ b.abs().T
    if extra is not None:
        want, size = want + extra, size + extra.abs()
    tol = (128 + -(-a.shape[1] // 128) + 4) * 2.0 ** -23 * size
    tol = tol + want.abs() * (2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -23) + 1e-38
    bad = ((got.double() - want).abs() > tol).sum().item()
    assert bad == 0, f"{bad} of {got.numel()} elements off"


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


SHAPES = [(1, 16, 16), (1, 1, 16), (1, 144, 4096), (7, 128, 128), (33, 272, 400), (128, 256, 128), (129, 257, 144),
          (300, 1000, 1040), (1000, 512, 2064), (2177, 768, 896)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_shapes(shape, block, out_dtype):
    fq = require_cuda()
    m, n, k = shape
    g = gen(m + n + k)
    kb = -(-k // 128)
    a, b = codes(g, (m, k), 0), codes(g, (n, k), 0)
    sa, sb = scales(g, (m, kb)), scales(g, (-(-n // block), kb))
    out = Guarded((m, n), out_dtype)
    fq.fp8q_matmul_blockwise(a, sa, b, sb, b_block=block, out_dtype=out_dtype, out=out.t)
    fq.check_device()
    out.check()
    check(out.t, values(a, sa, 0, 1), values(b, sb, 0, block))


@pytest.mark.parametrize("fa", [0, 1])
@pytest.mark.parametrize("fb", [0, 1])
@pytest.mark.parametrize("block", [1, 128])
def test_formats(fa, fb, block):
    fq = require_cuda()
    g = gen(10 + 2 * fa + fb)
    m, n, k = 200, 384, 656
    kb = -(-k // 128)
    a, b = codes(g, (m, k), fa), codes(g, (n, k), fb)
    sa, sb = scales(g, (m, kb)), scales(g, (-(-n // block), kb))
    y = fq.fp8q_matmul_blockwise(a, sa, b, sb, fa, fb, block, torch.float32)
    check(y, values(a, sa, fa, 1), values(b, sb, fb, block))


def test_every_code_once():
    """1 x 1 products of single codes: each finite code against each, one term a sum."""
    fq = require_cuda()
    for fmt in (0, 1):
        q = torch.arange(256, device="cuda", dtype=torch.uint8)
        q = q[torch.isfinite(q.view(FP8[fmt]).float())]
        a = torch.zeros(q.numel(), 16, dtype=torch.uint8, device="cuda")
        a[:, 3] = q
        one = torch.ones(q.numel(), 1, device="cuda")
        y = fq.fp8q_matmul_blockwise(a, one, a, one, fmt, fmt, 1, torch.float32)
        v = q.view(FP8[fmt]).double()
        assert torch.equal(y.double(), v[:, None] * v[None, :])


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("n", [256, 250])
def test_accumulate(block, n):
    fq = require_cuda()
    g = gen(3)
    m, k = 150, 400
    a, b = codes(g, (m, k), 1), codes(g, (n, k), 0)
    sa, sb = scales(g, (m, 4)), scales(g, (-(-n // block), 4))
    start = torch.randn(m, n, device="cuda", generator=g) * 1000
    out = start.clone()
    got = fq.fp8q_matmul_blockwise(a, sa, b, sb, 1, 0, block, torch.float32, accumulate=True, out=out)
    assert got is out
    check(out, values(a, sa, 1, 1), values(b, sb, 0, block), start.double())


def test_misaligned_out():
    """An output that starts 2 (4) bytes off a 32-byte line takes the element stores."""
    fq = require_cuda()
    g = gen(4)
    m, n, k = 130, 272, 272
    a, b = codes(g, (m, k), 0), codes(g, (n, k), 0)
    sa, sb = scales(g, (m, 3)), scales(g, (3, 3))
    for dt in (torch.bfloat16, torch.float32):
        raw = torch.full((m * n + 64,), 7.0, dtype=dt, device="cuda")
        out = raw[1:1 + m * n].view(m, n)
        fq.fp8q_matmul_blockwise(a, sa, b, sb, out_dtype=dt, out=out)
        check(out, values(a, sa, 0, 1), values(b, sb, 0, 128))
        assert raw[0].item() == 7.0 and (raw[1 + m * n:] == 7.0).all()


def test_nonfinite_codes_stay_in_their_row_and_column():
    fq = require_cuda()
    g = gen(5)
    m, n, k = 140, 270, 144
    a, b = codes(g, (m, k), 0), codes(g, (n, k), 0)
    a[17, 20], b[200, 143] = 0x7F, 0xFF
    one_a, one_b = torch.ones(m, 2, device="cuda"), torch.ones(3, 2, device="cuda")
    y = fq.fp8q_matmul_blockwise(a, one_a, b, one_b, out_dtype=torch.float32)
    bad = torch.isnan(y)
    want = torch.zeros_like(bad)
    want[17], want[:, 200] = True, True
    assert torch.equal(bad, want)
    a = codes(g, (m, k), 1) & 0x7F  # an E5M2 infinity times positive values
    a[3, 5] = 0x7C
    b = torch.full((n, k), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    y = fq.fp8q_matmul_blockwise(a, one_a, b, one_b, 1, 0, out_dtype=torch.float32)
    assert torch.isinf(y[3]).all() and torch.isfinite(y[:3]).all() and torch.isfinite(y[4:]).all()


def test_repeats_bit_for_bit():
    fq = require_cuda()
    g = gen(6)
    for m, n, k, block in ((1, 4096, 7168, 128), (777, 1296, 2064, 1)):
        kb = -(-k // 128)
        a, b = codes(g, (m, k), 0), codes(g, (n, k), 0)
        sa, sb = scales(g, (m, kb)), scales(g, (-(-n // block), kb))
        y = fq.fp8q_matmul_blockwise(a, sa, b, sb, b_block=block, out_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(y, fq.fp8q_matmul_blockwise(a, sa, b, sb, b_block=block, out_dtype=torch.float32))


def test_empty_reduction_and_empty_outputs():
    fq = require_cuda()
    a, b = (torch.empty(r, 0, dtype=torch.uint8, device="cuda") for r in (5, 48))
    sa, sb = torch.empty(5, 0, device="cuda"), torch.empty(1, 0, device="cuda")
    out = torch.full((5, 48), 3.0, device="cuda")
    fq.fp8q_matmul_blockwise(a, sa, b, sb, out_dtype=torch.float32, accumulate=True, out=out)
    assert (out == 3.0).all()
    fq.fp8q_matmul_blockwise(a, sa, b, sb, out_dtype=torch.float32, out=out)
    assert (out == 0.0).all()
    a, sa = torch.empty(0, 128, dtype=torch.uint8, device="cuda"), torch.empty(0, 1, device="cuda")
    b, sb = torch.zeros(48, 128, dtype=torch.uint8, device="cuda"), torch.ones(1, 1, device="cuda")
    assert fq.fp8q_matmul_blockwise(a, sa, b, sb).shape == (0, 48)


def test_output_beyond_31_bits():
    """More than 2^31 output elements; rows on both sides of the limit are checked."""
    fq = require_cuda()
    g = gen(7)
    m, n, k = 70001, 32768, 16
    a, b = codes(g, (m, k), 0), codes(g, (n, k), 0)
    sa, sb = scales(g, (m, 1)), scales(g, (n // 128, 1))
    y = fq.fp8q_matmul_blockwise(a, sa, b, sb)
    rows = torch.tensor([0, 1, 65535, 65536, 65537, 69999, 70000], device="cuda")
    check(y[rows], values(a[rows], sa[rows], 0, 1), values(b, sb, 0, 128))


def test_other_stream():
    """Inputs made on the default stream, product on another that waits for it."""
    fq = require_cuda()
    g = gen(8)
    s = torch.cuda.Stream()
    a, b = codes(g, (512, 4096), 0), codes(g, (1024, 4096), 0)
    sa, sb = scales(g, (512, 32)), scales(g, (8, 32))
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = fq.fp8q_matmul_blockwise(a, sa, b, sb)
    torch.cuda.current_stream().wait_stream(s)
    check(y, values(a, sa, 0, 1), values(b, sb, 0, 128))


def test_graph_capture():
    fq = require_cuda()
    g = gen(9)
    a, b = codes(g, (64, 2048), 0), codes(g, (512, 2048), 0)
    sa, sb = scales(g, (64, 16)), scales(g, (4, 16))
    out = torch.empty(64, 512, dtype=torch.bfloat16, device="cuda")
    fq.fp8q_matmul_blockwise(a, sa, b, sb, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.fp8q_matmul_blockwise(a, sa, b, sb, out=out)
    a.copy_(codes(g, (64, 2048), 0))
    graph.replay()
    check(out, values(a, sa, 0, 1), values(b, sb, 0, 128))


GROUPS = [[0, 128, 256], [0, 0, 1, 1, 130, 387, 387], [0, 5, 6, 7, 135], [3, 200, 200, 333], [0, 0, 0], [0, 1000]]


@pytest.mark.parametrize("offsets", GROUPS)
@pytest.mark.parametrize("nk", [(256, 256), (400, 1040), (250, 144), (16, 16)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_grouped(offsets, nk, out_dtype):
    """Groups that are empty, start anywhere, and leave rows before and after them alone."""
    fq = require_cuda()
    n, k = nk
    g = gen(sum(offsets) + n)
    rows, e, kb = offsets[-1] + 9, len(offsets) - 1, -(-k // 128)
    a, b = codes(g, (rows, k), 0), codes(g, (e, n, k), 0)
    sa, sb = scales(g, (rows, kb)), scales(g, (e, -(-n // 128), kb))
    out = Guarded((rows, n), out_dtype)
    out.t.fill_(7.0)
    fq.fp8q_matmul_grouped(a, sa, b, sb, offsets, out_dtype=out_dtype, out=out.t)
    fq.check_device()
    out.check()
    av = values(a, sa, 0, 1)
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        if hi > lo:
            check(out.t[lo:hi], av[lo:hi], values(b[i], sb[i], 0, 128))
    assert (out.t[:offsets[0]] == 7.0).all() and (out.t[offsets[-1]:] == 7.0).all()


def test_grouped_nan_rows_do_not_reach_other_groups():
    fq = require_cuda()
    g = gen(12)
    off, n, k = [0, 50, 100, 300], 256, 256
    a, b = codes(g, (300, k), 0), codes(g, (3, n, k), 0)
    a[50:100] = 0x7F
    b[1] = 0x7F
    sa, sb = scales(g, (300, 2)), scales(g, (3, 2, 2))
    y = fq.fp8q_matmul_grouped(a, sa, b, sb, off)
    assert torch.isnan(y[50:100]).all() and torch.isfinite(y[:50]).all() and torch.isfinite(y[100:]).all()


@pytest.mark.parametrize("experts", [1, 300, 4096])
def test_grouped_many_groups(experts):
    fq = require_cuda()
    g = gen(13)
    n, k = 64, 128
    count = torch.randint(0, 4, (experts,), generator=g, device="cuda")
    off = torch.cat([count.new_zeros(1), count.cumsum(0)])
    rows = int(off[-1])
    a, b = codes(g, (rows, k), 0), codes(g, (experts, n, k), 0)
    sa, sb = scales(g, (rows, 1)), scales(g, (experts, 1, 1))
    y = fq.fp8q_matmul_grouped(a, sa, b, sb, off, out_dtype=torch.float32)
    of = torch.repeat_interleave(torch.arange(experts, device="cuda"), count)
    av, bv = values(a, sa, 0, 1), values(b, sb, 0, 128)
    want = torch.einsum("rk,rnk->rn", av, bv[of])
    size = torch.einsum("rk,rnk->rn", av.abs(), bv[of].abs())
    assert ((y.double() - want).abs() <= 133 * 2.0 ** -23 * size + 2.0 ** -23 * want.abs()).all()


WGRAD_GROUPS = [[0, 128, 256], [0, 0, 128, 128, 640, 640], [0, 0, 0], [128, 256, 512], [0, 128, 144], [0, 1024]]


@pytest.mark.parametrize("offsets", WGRAD_GROUPS)
@pytest.mark.parametrize("mn", [(256, 256), (144, 400), (130, 250)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_grouped_wgrad(offsets, mn, out_dtype):
    fq = require_cuda()
    m, n = mn
    g = gen(sum(offsets) + n)
    e, rows = len(offsets) - 1, offsets[-1] + (0 if offsets[-1] % 128 else 32)
    rb = -(-rows // 128)
    a, b = codes(g, (m, rows), 1), codes(g, (n, rows), 0)
    sa, sb = scales(g, (m, rb)), scales(g, (n, rb))
    out = Guarded((e, m, n), out_dtype)
    fq.fp8q_matmul_grouped_wgrad(a, sa, b, sb, offsets, 1, 0, out_dtype, out=out.t)
    fq.check_device()
    out.check()
    av, bv = values(a, sa, 1, 1), values(b, sb, 0, 1)
    for i in range(e):
        lo, hi = offsets[i], offsets[i + 1]
        check(out.t[i], av[:, lo:hi], bv[:, lo:hi])
    if out_dtype == torch.float32:
        start = torch.randn(e, m, n, device="cuda", generator=g)
        got = start.clone()
        fq.fp8q_matmul_grouped_wgrad(a, sa, b, sb, offsets, 1, 0, accumulate=True, out=got)
        for i in range(e):
            lo, hi = offsets[i], offsets[i + 1]
            check(got[i], av[:, lo:hi], bv[:, lo:hi], start[i].double())


def test_linear_layer_with_the_quantizer():
    """Fprop, Dgrad and Wgrad of one layer from fp8q_quantize_blockwise's copies: within the
    quantization error of the BF16 products.  Each factor is rounded to 3 (2) mantissa bits, half a
    unit is 2^-4 (2^-3) of a value, so a product of independent values is off by less than
    sqrt(2^-8 + 2^-8) (sqrt(2^-6 + 2^-8)) in the norm, times 1.1 for the sampling."""
    fq = require_cuda()
    g = gen(14)
    t, n, k = 400, 528, 784
    x = torch.randn(t, k, device="cuda", generator=g).bfloat16()
    w = (0.05 * torch.randn(n, k, device="cuda", generator=g)).bfloat16()
    dy = (0.01 * torch.randn(t, n, device="cuda", generator=g)).bfloat16()
    qx = fq.fp8q_quantize_blockwise(x, fq.E4M3, fq.BLOCK_1X128, direction=fq.BOTH)
    qw = fq.fp8q_quantize_blockwise(w, fq.E4M3, fq.BLOCK_128X128, direction=fq.BOTH)
    qd = fq.fp8q_quantize_blockwise(dy, fq.E5M2, fq.BLOCK_1X128, direction=fq.BOTH)
    y = fq.fp8q_matmul_blockwise(qx["q"], qx["scale_inv"], qw["q"], qw["scale_inv"])
    dx = fq.fp8q_matmul_blockwise(qd["q"], qd["scale_inv"], qw["q_t"], qw["scale_inv_t"], fq.E5M2)
    dw = fq.fp8q_matmul_blockwise(qd["q_t"], qd["scale_inv_t"], qx["q_t"], qx["scale_inv_t"], fq.E5M2, fq.E4M3,
                                  fq.BLOCK_1X128, torch.float32)
    for got, want, bound in ((y, x.double() @ w.double().T, (2 ** -8 + 2 ** -8) ** 0.5),
                             (dx, dy.double() @ w.double(), (2 ** -6 + 2 ** -8) ** 0.5),
                             (dw, dy.double().T @ x.double(), (2 ** -6 + 2 ** -8) ** 0.5)):
        assert (got.double() - want).norm() / want.norm() < 1.1 * bound


def test_python_checks():
    fq = require_cuda()
    a = torch.zeros(4, 32, dtype=torch.uint8, device="cuda")
    s = torch.ones(4, 1, device="cuda")
    one = torch.ones(1, 1, device="cuda")
    mm = fq.fp8q_matmul_blockwise
    for bad in (lambda: mm(a.float(), s, a, one), lambda: mm(a.t(), s, a, one), lambda: mm(a, s, a[:, :16].contiguous(), one),
                lambda: mm(a, s[:3], a, one), lambda: mm(a, s, a, s), lambda: mm(a, s.double(), a, one),
                lambda: mm(a, s, a, one, accumulate=True, out_dtype=torch.float32),
                lambda: mm(a, s, a, one, out=torch.empty(4, 5, dtype=torch.bfloat16, device="cuda")),
                lambda: fq.fp8q_matmul_grouped(a, s, a[None], one[None], [0, 2, 4]),
                lambda: fq.fp8q_matmul_grouped(a, s, a[None], one[None], None)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        mm(a, s, a, one, out_dtype=torch.float16)
    with pytest.raises(fq.Fp8qError, match="multiple of 16"):
        b = torch.zeros(4, 24, dtype=torch.uint8, device="cuda")
        mm(b, s, b, one)
    with pytest.raises(fq.Fp8qError, match="FP32"):
        mm(a, s, a, one, accumulate=True, out=torch.empty(4, 4, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("m,n,k", [(1, 512, 2048), (130, 256, 16384), (700, 8192, 1024)])
def test_waits_run_out_and_are_reported(m, n, k):
    """Without loads every wait ends after the budget, whatever the form (split, one CTA, pairs): the call
    returns, the failure is reported, nothing is written outside the output, and the next call is right."""
    fq = require_cuda()
    g = gen(m)
    kb = k // 128
    a, b = codes(g, (m, k), 0), codes(g, (n, k), 0)
    sa, sb = scales(g, (m, kb)), scales(g, (n // 128, kb))
    out = Guarded((m, n), torch.float32)
    try:
        fq.set_wait_budget_ns(20_000_000)
        fq.debug_stall_matmul_loads(True)
        fq.fp8q_matmul_blockwise(a, sa, b, sb, out_dtype=torch.float32, out=out.t)
        with pytest.raises(fq.Fp8qError, match="gave up"):
            fq.check_device()
    finally:
        fq.debug_stall_matmul_loads(False)
        fq.set_wait_budget_ns(1_000_000_000)
    out.check()
    fq.fp8q_matmul_blockwise(a, sa, b, sb, out_dtype=torch.float32, out=out.t)
    fq.check_device()
    check(out.t, values(a, sa, 0, 1), values(b, sb, 0, 128))
