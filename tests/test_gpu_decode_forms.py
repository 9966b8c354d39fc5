"""The few-token expert layer where four warps share a unit of the first product over several rounds of K, the last
of which most of them have no block for.  The bounds are those of test_gpu_decode.py."""
import pytest
import torch

from gpu_util import require_cuda
from test_gpu_decode import case, check

pytestmark = pytest.mark.gpu


def four_warps(tokens, top, experts, hidden, inner):
    """The first kernel's rule: blocks of K leave many of 8 warps idle, and there are units enough."""
    blocks, idle = -(-hidden // 128), lambda w: -(-hidden // 128) % w and w - -(-hidden // 128) % w  # noqa: E731
    units = min(tokens * top, experts) * -(-inner // 128) * 4
    return 8 * (idle(8) - idle(4)) > blocks and units >= 8 * torch.cuda.get_device_properties(0).multi_processor_count


# 17, 9, 9, 10 (with 4 warps: 2 idle in the last round) and 25 blocks of K
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("tokens,top,experts,hidden,inner", [
    (61, 6, 40, 2064, 1360), (64, 8, 64, 1152, 1008), (11, 8, 96, 1040, 1024), (64, 32, 48, 1280, 912), (5, 8, 64, 3104, 1264)])
def test_four_warps_a_unit(tokens, top, experts, hidden, inner, fmt):
    fq = require_cuda()
    assert four_warps(tokens, top, experts, hidden, inner)
    for out_dtype in (torch.float32, torch.bfloat16):
        check(fq, *case(tokens, top, experts, hidden, inner, fmt, tokens + inner), out_dtype)


def test_four_warps_dropped_and_repeated_slots():
    """Experts with no, one and many tokens, and fewer units than the slots allow for."""
    fq = require_cuda()
    c = case(61, 6, 40, 2064, 1360, 0, 3)
    ids = c[1]
    ids[ids % 3 == 1] = -1
    ids[7], ids[8, 2], ids[40:, 0] = -1, 1000, 5
    check(fq, *c)
