"""The expert layer for a few tokens rejects bad arguments on the host, before any CUDA call."""
import ctypes

import pytest

import mxfp8_quantization_amax_gb300 as fq


@pytest.fixture(scope="module")
def lib():
    fq.build()
    return fq.lib()


def test_decode(lib):
    buf = ctypes.create_string_buffer(256)
    a = (ctypes.addressof(buf) + 31) // 32 * 32
    need = lib.fp8q_moe_decode_workspace_bytes(4, 2, 48)
    assert need >= 8 * 128 * 4 and lib.fp8q_moe_decode_workspace_bytes(65, 2, 48) == 0 and lib.fp8q_moe_decode_workspace_bytes(0, 2, 48) == 0
    base = dict(x=a, tokens=4, hidden=32, inner=48, experts=8, top_k=2, ids=a, w=a, w1=a, s1=a, w2=a, s2=a, fmt=0, odt=0, out=a, ws=a, bytes=need)
    for change, status in [
            (dict(tokens=-1), 1), (dict(tokens=65), 2), (dict(hidden=0), 1), (dict(inner=0), 1), (dict(hidden=24), 2), (dict(inner=40), 2),
            (dict(experts=0), 1), (dict(experts=1025), 2), (dict(top_k=0), 2), (dict(top_k=33), 2), (dict(fmt=2), 1), (dict(odt=2), 1),
            (dict(x=None), 1), (dict(x=a + 8), 1), (dict(ids=None), 1), (dict(ids=a + 2), 1), (dict(w=None), 1), (dict(w1=None), 1),
            (dict(w1=a + 8), 1), (dict(w2=a + 8), 1), (dict(s1=None), 1), (dict(s2=a + 2), 1), (dict(out=None), 1), (dict(out=a + 1), 1),
            (dict(odt=1, out=a + 2), 1), (dict(ws=None), 1), (dict(ws=a + 8), 1), (dict(bytes=need - 1), 1), (dict(hidden=2**21), 2),
            (dict(tokens=0, x=None, out=None, ws=None), 0)]:
        v = dict(base)
        v.update(change)
        assert lib.fp8q_moe_decode(*v.values(), None) == status, change
