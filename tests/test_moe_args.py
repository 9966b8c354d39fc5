"""The entry points of the expert layer reject bad arguments on the host, before any CUDA call."""
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


def test_route(lib, a):
    base = dict(x=a, dt=1, tokens=4, experts=64, top_k=8, score=0, bias=None, groups=8, top_groups=4, renorm=1, scale=1.0, w=a, ids=a)
    refused(lib.fp8q_moe_route, base, [
        (dict(dt=2), 1), (dict(tokens=-1), 1), (dict(experts=0), 1), (dict(experts=1025, groups=1, top_groups=1), 2), (dict(top_k=0), 1),
        (dict(top_k=65), 1), (dict(top_k=33), 2), (dict(score=2), 1), (dict(bias=a + 2), 1), (dict(groups=0), 1), (dict(groups=7), 1),
        (dict(groups=64), 1), (dict(top_groups=0), 1), (dict(top_groups=9), 1), (dict(top_groups=1, top_k=9), 1), (dict(x=None), 1),
        (dict(x=a + 2), 1), (dict(x=a + 1, dt=0), 1), (dict(w=None), 1), (dict(ids=a + 1), 1), (dict(tokens=0, x=None, w=None), 0)])


def test_route_backward(lib, a):
    base = dict(x=a, dt=0, tokens=4, experts=64, top_k=8, score=1, renorm=1, scale=1.0, ids=a, d=a, dx=a)
    refused(lib.fp8q_moe_route_backward, base, [
        (dict(dt=3), 1), (dict(score=-1), 1), (dict(ids=None), 1), (dict(d=a + 2), 1), (dict(dx=None), 1), (dict(dx=a + 1), 1),
        (dict(top_k=65), 1), (dict(tokens=0, ids=None), 0)])


def test_rows_and_workspace(lib):
    assert lib.fp8q_moe_rows(0, 8, 128) == 0
    assert lib.fp8q_moe_rows(1, 8, 128) == 128
    assert lib.fp8q_moe_rows(128, 64, 1) == 128
    assert lib.fp8q_moe_rows(1000, 8, 128) == (1000 + 8 * 127) // 128 * 128
    assert lib.fp8q_moe_rows(-1, 8, 1) == -1 and lib.fp8q_moe_rows(1, 0, 1) == -1 and lib.fp8q_moe_rows(1, 1, 0) == -1
    assert lib.fp8q_moe_plan_workspace_bytes(4097, 64) >= 256
    assert lib.fp8q_moe_plan_workspace_bytes(-1, 64) == 0


def test_plan(lib, a):
    base = dict(ids=a, slots=16, experts=8, align=1, rows=16, offsets=a, row_of=a, src=a, ws=a, ws_bytes=1 << 20)
    refused(lib.fp8q_moe_plan, base, [
        (dict(slots=-1), 1), (dict(experts=0), 1), (dict(experts=1025), 2), (dict(align=0), 1), (dict(align=5000), 1), (dict(rows=15), 1),
        (dict(align=128), 1), (dict(offsets=None), 1), (dict(offsets=a + 4), 1), (dict(ids=None), 1), (dict(row_of=a + 1), 1),
        (dict(src=None), 1), (dict(slots=5000, rows=5000, ws=None), 1), (dict(slots=5000, rows=5000, ws_bytes=8), 1), (dict(slots=2**31, rows=2**31), 2), (dict(rows=2**31), 2)])


def test_dispatch(lib, a):
    base = dict(x=a, dt=0, tokens=4, cols=32, k=2, src=a, rows=16, fmt=0, pow2=0, dir=3, q=a, s=a, qt=a, st=a)
    refused(lib.fp8q_moe_dispatch, base, [
        (dict(dt=1), 2), (dict(dt=5), 1), (dict(fmt=2), 1), (dict(dir=0), 1), (dict(tokens=-1), 1), (dict(k=0), 1), (dict(cols=24), 2),
        (dict(rows=8), 2), (dict(x=None), 1), (dict(x=a + 8), 1), (dict(src=None), 1), (dict(q=None), 1), (dict(qt=a + 8), 1),
        (dict(st=None), 1), (dict(rows=0, x=None, src=None), 0), (dict(rows=2**31), 2), (dict(cols=2**24), 2)])


def test_combine(lib, a):
    base = dict(y=a, dt=0, rows=8, cols=32, row_of=a, w=None, tokens=4, k=2, out=a)
    refused(lib.fp8q_moe_combine, base, [
        (dict(dt=2), 1), (dict(rows=-1), 1), (dict(k=0), 2), (dict(k=33), 2), (dict(y=None), 1), (dict(y=a + 1), 1), (dict(out=None), 1),
        (dict(row_of=None), 1), (dict(w=a + 2), 1), (dict(tokens=0, y=None, out=None), 0)])
    base = dict(d=a, y=a, dt=1, rows=8, cols=32, row_of=a, src=a, w=a, tokens=4, k=2, dy=a, dw=a)
    refused(lib.fp8q_moe_combine_backward, base, [
        (dict(dt=2), 1), (dict(d=None), 1), (dict(y=a + 2), 1), (dict(dy=None), 1), (dict(src=None), 1), (dict(w=None), 1),
        (dict(dw=None), 1), (dict(row_of=a + 2), 1), (dict(k=33), 2), (dict(tokens=0, rows=0, d=None, y=None, src=None), 0)])
