"""The clip refuses outputs that overlap another tensor, on the host: what would be read after it was written."""
import ctypes

import pytest

import mxfp8_quantization_amax_gb300 as fq

BF16, FP32 = 0, 1
A = 1 << 20  # an address; nothing is read or written


@pytest.fixture(scope="module")
def lib():
    fq.build()
    return fq.lib()


def status(lib, grads, sizes, dts, out):
    n = len(grads)
    need = lib.fp8q_clip_grads_workspace_bytes(n)
    arrays = [(t * n)(*v) for t, v in ((ctypes.c_void_p, grads), (ctypes.c_int64, sizes), (ctypes.c_int32, dts), (ctypes.c_void_p, out))]
    return lib.fp8q_clip_grads(*arrays[:3], n, 1.0, arrays[3], A, A, A, need, None)


@pytest.mark.parametrize("grads,sizes,dts,out", [
    ([A, A + 400], [100, 100], [FP32, FP32], [A + 400, A]),                     # each into the other's place
    ([A, A], [100, 100], [FP32, FP32], [A + 4000, A]),                          # a gradient twice, once in place
    ([A, A], [100, 100], [FP32, FP32], [A, A]),
    ([A], [100], [FP32], [A + 4]),                                              # one value on
    ([A + 4], [100], [FP32], [A]),
    ([A, A + 4000], [100, 100], [FP32, BF16], [A + 8000, A + 8000 + 398]),      # two outputs
    ([A, A + 198], [100, 100], [BF16, BF16], [A, A + 198]),                     # both in place
    ([A, A + 4000, A + 9000], [1000, 1, 1], [FP32, FP32, FP32], [A, A + 3996, A + 9000]),  # inside a long one
    ([A + 4 * i for i in range(300)], [1] * 300, [FP32] * 300, [A + 4 * (i + 1) for i in range(300)]),
])
def test_overlap_is_refused(lib, grads, sizes, dts, out):
    assert status(lib, grads, sizes, dts, out) == 1
    assert b"overlap" in lib.fp8q_last_error_string()
