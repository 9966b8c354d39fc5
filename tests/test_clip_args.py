"""The gradients' norm and clip reject bad arguments on the host, before any CUDA call."""
import ctypes

import pytest

import mxfp8_quantization_amax_gb300 as fq


@pytest.fixture(scope="module")
def lib():
    fq.build()
    return fq.lib()


def test_clip(lib):
    buf = ctypes.create_string_buffer(256)
    a = (ctypes.addressof(buf) + 31) // 32 * 32
    P, I64, I32 = ctypes.c_void_p * 2, ctypes.c_int64 * 2, ctypes.c_int32 * 2
    need = lib.fp8q_clip_grads_workspace_bytes(2)
    assert 0 < need < 1 << 16 and lib.fp8q_clip_grads_workspace_bytes(-1) == 0
    assert lib.fp8q_clip_grads_workspace_bytes(1000) > need
    base = dict(g=P(a, a), n=I64(4, 4), dt=I32(0, 1), count=2, most=1.0, out=P(a, a), norm=a, scale=a, ws=a, bytes=need)
    for change, status in [
            (dict(count=-1), 1), (dict(count=2**21), 1), (dict(g=None), 1), (dict(n=None), 1), (dict(dt=None), 1), (dict(dt=I32(0, 2)), 1),
            (dict(n=I64(4, -1)), 1), (dict(n=I64(4, 2**43)), 2), (dict(n=I64(2**41 + 2**40, 2**41)), 2), (dict(g=P(a, None)), 1), (dict(g=P(a, a + 2)), 1),
            (dict(g=P(a + 1, a)), 1), (dict(out=P(None, a)), 1), (dict(out=P(a, a + 2)), 1), (dict(norm=None), 1), (dict(norm=a + 2), 1),
            (dict(scale=None), 1), (dict(scale=a + 1), 1), (dict(most=-1.0), 1), (dict(most=float("nan")), 1), (dict(ws=None), 1),
            (dict(ws=a + 4), 1), (dict(bytes=need - 1), 1)]:
        v = dict(base)
        v.update(change)
        assert lib.fp8q_clip_grads(*v.values(), None) == status, change
