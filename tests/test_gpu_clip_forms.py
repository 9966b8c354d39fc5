"""The gradients' norm and clip with more partial sums than the writing CTAs add up themselves, with nothing to add
up, and with lists of every sort of place.  The bounds are those of test_gpu_clip.py."""
import pytest
import torch

from gpu_util import require_cuda
from test_gpu_clip import BF16, FP32, check, tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [4864, 4865, 6000])
def test_many_tensors(count):
    """One partial sum each: 4 * 1216 = 4864 of them are the most that every writing CTA adds up."""
    fq = require_cuda()
    g = tensors([3 + i % 5 for i in range(count)], (FP32, BF16), count)
    norm = sum(float(t.double().square().sum()) for t in g) ** 0.5
    check(fq.fp8q_clip_grads(g, norm / 3), g, norm / 3)
    keep = [t.clone() for t in g]
    check(fq.fp8q_clip_grads(g, norm / 2, out=g), keep, norm / 2)


def test_nothing_but_empty_tensors():
    fq = require_cuda()
    g = [torch.empty(0, device="cuda"), torch.empty(3, 0, device="cuda", dtype=BF16)]
    r = fq.fp8q_clip_grads(g, 1.0)
    assert float(r["norm"]) == 0.0 and float(r["scale"]) == 1.0 and [t.shape for t in r["grads"]] == [t.shape for t in g]
    assert float(fq.fp8q_grad_norm(g)) == 0.0


def test_outputs_side_by_side():
    """Neighbours, empty tensors in others' places and gradients that share memory are no overlap; swapped places are."""
    fq = require_cuda()
    base, out = torch.randn(3000, device="cuda"), torch.empty(3000, device="cuda")
    g = [base[:1000], base[1000:1001], base[500:500], base[1001:]]
    check(fq.fp8q_clip_grads(g, 1.0, out=[out[:1000], out[1000:1001], out[5:5], out[1001:]]), g, 1.0)
    shared = [base[:2000], base[1000:]]
    check(fq.fp8q_clip_grads(shared, 1.0, out=[out[:2000], torch.empty_like(shared[1])]), shared, 1.0)
    for outs in ([g[3], g[1], g[2], g[0]], [shared[0], shared[1]]):
        with pytest.raises((fq.Fp8qError, ValueError)):
            fq.fp8q_clip_grads(g if len(outs) == 4 else shared, 1.0, out=outs)
    keep = [t.clone() for t in g]
    check(fq.fp8q_clip_grads(g, 1.0, out=g), keep, 1.0)
