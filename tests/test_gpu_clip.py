"""The gradients' norm and clip against 64 bits.

With u = 2^-24: a thread adds at most 64 squares in a row in FP32 (and four such sums), the rest is FP64, so
the sum of squares is off by 67 u and the norm by 34 u and its rounding; the scale takes an addition and a
division, a value one product and its type's rounding."""
import pytest
import torch

from gpu_util import Guarded, require_cuda

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NORM, SCALE = 36 * U, 40 * U
BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, FP32: U}


def tensors(sizes, dtypes, seed, spread=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(spread * (1 + i % 3) * torch.randn(n, device="cuda", generator=g)).to(dtypes[i % len(dtypes)]) for i, n in enumerate(sizes)]


def check(r, before, max_norm):
    norm = sum(float(g.double().square().sum()) for g in before) ** 0.5
    scale = min(1.0, max_norm / (norm + 1e-6))
    assert abs(float(r["norm"]) - norm) <= NORM * norm
    assert abs(float(r["scale"]) - scale) <= SCALE * scale
    for g, o in zip(before, r["grads"]):
        assert o.dtype == g.dtype and o.shape == g.shape
        want = g.double() * scale
        assert ((o.double() - want).abs() <= want.abs() * (HALF[g.dtype] + SCALE + 2 * U) * (1 + 2.0 ** -7) + 1e-40).all()


SIZES = [[1], [0, 5, 0], [7, 8, 9, 16383, 16384, 16385], [1000003, 3, 40000], [3] * 600, [8192 * 5, 1, 300000]]


@pytest.mark.parametrize("dtypes", [(BF16,), (FP32,), (BF16, FP32)])
@pytest.mark.parametrize("sizes", SIZES, ids=[str(len(s)) + "x" + str(s[0]) for s in SIZES])
def test_clip(sizes, dtypes):
    fq = require_cuda()
    g = tensors(sizes, dtypes, len(sizes))
    norm = sum(float(t.double().square().sum()) for t in g) ** 0.5
    for over in (0.5, 3.0):
        check(fq.fp8q_clip_grads(g, norm / over), g, norm / over)
        keep = [t.clone() for t in g]
        inside = [t.clone() for t in g]
        r = fq.fp8q_clip_grads(inside, norm / over, out=inside)
        assert all(a is b for a, b in zip(r["grads"], inside))
        check(r, keep, norm / over)
        if over < 1:
            assert float(r["scale"]) == 1.0 and all(torch.equal(a, b) for a, b in zip(inside, keep))
    assert torch.equal(fq.fp8q_grad_norm(g), r["norm"]) and all(torch.equal(a, b) for a, b in zip(g, keep))


def test_large_sum():
    """3 * 2^26 values: a sum in FP32 alone would lose digits."""
    fq = require_cuda()
    g = [torch.full((3 * 2 ** 25,), 0.1, device="cuda"), torch.full((3 * 2 ** 25 + 1,), 0.1, device="cuda", dtype=BF16)]
    check(fq.fp8q_clip_grads(g, 1.0, out=g), [torch.full_like(t, 0.1) for t in g], 1.0)


def test_past_32_bits():
    fq = require_cuda()
    g = torch.zeros(2 ** 32 + 5, device="cuda", dtype=BF16)
    g[-1], g[2 ** 31] = 3.0, 4.0
    r = fq.fp8q_clip_grads([g], 1.0, out=[g])
    assert abs(float(r["norm"]) - 5.0) < 1e-6 and abs(float(g[-1]) - 0.6) < 0.6 * 2 ** -8 and abs(float(g[2 ** 31]) - 0.8) < 0.8 * 2 ** -8


def test_unaligned_and_guards():
    fq = require_cuda()
    base = tensors([50021], (BF16,), 5)[0]
    g = [base[1:30002], base[30003:50000]]
    out = [Guarded((30001,), BF16), Guarded((19997,), BF16)]
    check(fq.fp8q_clip_grads(g, 0.3, out=[o.t for o in out]), g, 0.3)
    for o in out:
        o.check()
    shaped = [torch.randn(5, 7, 11, device="cuda"), torch.randn((), device="cuda")]
    check(fq.fp8q_clip_grads(shaped, 0.3), shaped, 0.3)


def test_nonfinite():
    """What the formula gives: Inf in the norm makes the scale 0, NaN makes it NaN."""
    fq = require_cuda()
    g = tensors([1000, 77], (FP32,), 6)
    g[1][5] = float("inf")
    r = fq.fp8q_clip_grads(g, 1.0)
    assert float(r["norm"]) == float("inf") and float(r["scale"]) == 0.0 and (r["grads"][0] == 0).all() and torch.isnan(r["grads"][1][5])
    g[0][3] = float("nan")
    r = fq.fp8q_clip_grads(g, 1.0)
    assert torch.isnan(r["norm"]).all() and torch.isnan(r["scale"]).all() and torch.isnan(r["grads"][0]).all()
    zero = [torch.zeros(10, device="cuda")]
    r = fq.fp8q_clip_grads(zero, 1.0)
    assert float(r["norm"]) == 0.0 and float(r["scale"]) == 1.0
    assert float(fq.fp8q_clip_grads(tensors([10], (FP32,), 1), 0.0)["scale"]) == 0.0


def test_same_bits_on_streams_and_in_graphs():
    fq = require_cuda()
    g = tensors([300000, 17, 65536], (FP32, BF16), 7)
    want = fq.fp8q_clip_grads(g, 0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = fq.fp8q_clip_grads(g, 0.5)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got["norm"], want["norm"]) and all(torch.equal(a, b) for a, b in zip(got["grads"], want["grads"]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = fq.fp8q_clip_grads(g, 0.5)
    for i in range(2):
        for a, b in zip(g, tensors([300000, 17, 65536], (FP32, BF16), 10 + i)):
            a.copy_(b)
        graph.replay()
        now = fq.fp8q_clip_grads(g, 0.5)
        assert torch.equal(held["scale"], now["scale"]) and all(torch.equal(a, b) for a, b in zip(held["grads"], now["grads"]))


def test_refusals():
    fq = require_cuda()
    a = torch.randn(8, 8, device="cuda")
    for call in (lambda: fq.fp8q_clip_grads([], 1.0), lambda: fq.fp8q_clip_grads([a.half()], 1.0), lambda: fq.fp8q_clip_grads([a[:, :4]], 1.0),
                 lambda: fq.fp8q_clip_grads([a, a.cpu()], 1.0), lambda: fq.fp8q_clip_grads([a], 1.0, out=[]),
                 lambda: fq.fp8q_clip_grads([a, a], 1.0, out=[a, a]), lambda: fq.fp8q_clip_grads([a], 1.0, out=[a.bfloat16()]), lambda: fq.fp8q_grad_norm([a.cpu()])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_clip_grads([a], -1.0)
    empty = torch.empty(0, device="cuda")  # nothing of it is written
    assert float(fq.fp8q_clip_grads([empty, a, empty], 1.0, out=[empty, a.clone(), empty])["scale"]) < 1
    # a gradient twice counts twice
    twice = fq.fp8q_grad_norm([a, a])
    assert abs(float(twice) - 2 ** 0.5 * float(fq.fp8q_grad_norm([a]))) <= 2 ** -22 * float(twice)
