"""The product entry points reject bad arguments on the host, before any CUDA call."""
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


def dense(lib, buf, **kw):
    v = dict(a=buf, sa=buf, fa=0, b=buf, sb=buf, fb=0, block=128, m=4, n=32, k=32, dt=0, acc=0, out=buf)
    v.update(kw)
    return lib.fp8q_matmul_blockwise(*v.values(), None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(fa=2), 1, b"a_fmt"), (dict(fb=-1), 1, b"b_fmt"), (dict(block=64), 1, b"b_block"), (dict(dt=2), 1, b"out_dt"),
    (dict(acc=1), 2, b"FP32"), (dict(m=-1), 1, b">= 0"), (dict(k=24), 2, b"multiple of 16"), (dict(n=2**31), 2, b"large"),
    (dict(k=2**31), 2, b"large"), (dict(a=None), 1, b"a and b"), (dict(b=None), 1, b"a and b"), (dict(sa=None), 1, b"scales"),
    (dict(sb=None), 1, b"scales"), (dict(out=None), 1, b"out"),
])
def test_dense_refusals(lib, a, kw, status, word):
    assert dense(lib, a, **kw) == status
    assert word in lib.fp8q_last_error_string()


def test_alignment_refusals(lib, a):
    for kw in (dict(a=a + 8), dict(b=a + 8), dict(sa=a + 2), dict(sb=a + 2), dict(out=a + 1), dict(out=a + 2, dt=1)):
        assert dense(lib, a, **kw) == 1


def test_empty_outputs_do_nothing(lib, a):
    assert dense(lib, a, m=0, a=None, sa=None, out=None) == 0
    assert dense(lib, a, n=0, b=None, sb=None, out=None) == 0


def test_grouped_refusals(lib, a):
    def call(off=a, groups=2, rows=4, n=32, k=32, dt=0, out=a):
        return lib.fp8q_matmul_grouped(a, a, 0, a, a, 0, off, groups, rows, n, k, dt, out, None)

    assert call(off=None) == 1 and call(off=a + 4) == 1
    assert call(groups=0) == 1 and call(groups=5000) == 1
    assert call(k=8) == 2 and call(dt=3) == 1 and call(out=None) == 1
    assert call(n=2**30, groups=4) == 2
    assert call(rows=0, out=None) == 0


def test_wgrad_refusals(lib, a):
    def call(off=a, groups=2, rows=128, m=4, n=32, dt=1, acc=0, out=a):
        return lib.fp8q_matmul_grouped_wgrad(a, a, 0, a, a, 0, off, groups, rows, m, n, dt, acc, out, None)

    assert call(off=None) == 1 and call(rows=120) == 2 and call(groups=0) == 1
    assert call(dt=0, acc=1) == 2 and call(out=a + 2) == 1
    assert call(m=0, out=None) == 0
