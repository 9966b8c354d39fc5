"""The norm and the gated activation reject bad arguments on the host, before any CUDA call."""
import ctypes

import pytest

import mxfp8_quantization_amax_gb300 as fq


@pytest.fixture(scope="module")
def lib():
    fq.build()
    return fq.lib()


@pytest.fixture(scope="module")
def a():
    buf = ctypes.create_string_buffer(256)
    yield (ctypes.addressof(buf) + 31) // 32 * 32


def refused(fn, base, cases):
    for change, status in cases:
        v = dict(base)
        v.update(change)
        assert fn(*v.values(), None) == status, change


def test_rmsnorm(lib, a):
    base = dict(x=a, dt=0, residual=a, rdt=0, weight=a, wdt=1, rows=16, cols=32, eps=1e-6, fmt=0, dir=3, pow2=0, h=a, rstd=a, y=a,
                q=a, s=a, qt=a, st=a)
    nan, inf = float("nan"), float("inf")
    refused(lib.fp8q_rmsnorm, base, [
        (dict(dt=2), 1), (dict(rdt=2), 1), (dict(wdt=-1), 1), (dict(rows=-1), 1), (dict(cols=0), 1), (dict(cols=32769, dir=0), 2),
        (dict(rows=2**31), 2), (dict(eps=-1.0), 1), (dict(eps=nan), 1), (dict(eps=inf), 1), (dict(fmt=2), 1), (dict(dir=4), 1),
        (dict(dir=-1), 1), (dict(cols=24), 2), (dict(rows=8), 2), (dict(x=None), 1), (dict(x=a + 8), 1), (dict(residual=a + 2), 1),
        (dict(h=None), 1), (dict(h=a + 8), 1), (dict(weight=None), 1), (dict(weight=a + 4), 1), (dict(rstd=None), 1), (dict(rstd=a + 2), 1),
        (dict(y=a + 8), 1), (dict(q=None), 1), (dict(q=a + 8), 1), (dict(s=None), 1), (dict(qt=None), 1), (dict(st=a + 2), 1),
        (dict(dir=0, x=a + 1), 1), (dict(dir=0, y=a + 1), 1), (dict(dir=0, weight=a + 2), 1), (dict(rows=0, x=None, weight=None), 0)])


def test_rmsnorm_backward(lib, a):
    need = lib.fp8q_rmsnorm_backward_workspace_bytes(16, 32)
    assert need >= 16 * 32 * 4 and lib.fp8q_rmsnorm_backward_workspace_bytes(0, 32) == 0
    assert lib.fp8q_rmsnorm_backward_workspace_bytes(10**6, 7168) <= 700 * 7168 * 4
    assert lib.fp8q_rmsnorm_backward_workspace_bytes(4, 40000) == 0
    base = dict(dy=a, dt=0, h=a, hdt=1, weight=a, wdt=0, rstd=a, dh=None, rows=16, cols=32, dx=a, dw=a, ws=a, bytes=need)
    refused(lib.fp8q_rmsnorm_backward, base, [
        (dict(dt=2), 1), (dict(hdt=3), 1), (dict(wdt=9), 1), (dict(rows=-1), 1), (dict(cols=0), 1), (dict(cols=40000), 2), (dict(dy=None), 1),
        (dict(dy=a + 1), 1), (dict(h=None), 1), (dict(h=a + 2), 1), (dict(dh=a + 2), 1), (dict(dx=None), 1), (dict(weight=None), 1),
        (dict(weight=a + 1), 1), (dict(rstd=None), 1), (dict(dw=None), 1), (dict(dw=a + 2), 1), (dict(ws=None), 1), (dict(ws=a + 4), 1),
        (dict(bytes=need - 1), 1), (dict(rows=0, dw=None), 1)])


@pytest.mark.parametrize("backward", [False, True])
def test_swiglu(lib, a, backward):
    base = dict(h=a, da=a, dt=0, rows=16, inner=32, fmt=1, dir=3, pow2=0, dense=None, q=a, s=a, qt=a, st=a)
    fn = lib.fp8q_swiglu_backward
    if not backward:
        del base["da"]
        fn = lib.fp8q_swiglu
    cases = [(dict(dt=2), 1), (dict(rows=-1), 1), (dict(inner=-1), 1), (dict(fmt=3), 1), (dict(dir=5), 1), (dict(dir=0), 1),
             (dict(inner=12), 2), (dict(rows=9), 2), (dict(rows=2**31), 2), (dict(h=None), 1), (dict(h=a + 8), 1), (dict(dense=a + 8), 1),
             (dict(q=None), 1), (dict(qt=a + 8), 1), (dict(s=a + 1), 1), (dict(st=None), 1), (dict(dir=0, dense=a, h=a + 1), 1),
             (dict(rows=0, h=None), 0), (dict(inner=0, h=None, q=None), 0)]
    if backward:
        cases += [(dict(da=None), 1), (dict(da=a + 8), 1), (dict(inner=20), 2)]
    else:
        cases += [(dict(inner=24), 2)]
    refused(fn, base, cases)
