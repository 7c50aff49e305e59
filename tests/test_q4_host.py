"""CPU tests of the 4-bit cache's host rules: creation, the calls that do not
apply, and the arguments of kvc_read.  Buffer pointers are fake; every call
fails its checks before any CUDA call, or is host-only."""

import ctypes

import numpy as np
import pytest

from gqa_attention_preallocated_gb300 import _lib
from gqa_attention_preallocated_gb300.build import build_library

I32P = ctypes.POINTER(ctypes.c_int32)
I64P = ctypes.POINTER(ctypes.c_int64)
ARG, SHAPE, OVERFLOW = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    build_library()
    return _lib.lib()


def _bufs(layers, n, base=1 << 40):
    return [(ctypes.c_void_p * layers)(*[base + (j * layers + i) * (1 << 30) for i in range(layers)]) for j in range(n)]


def _create(L, layers=1, B=2, Hkv=2, max_len=64, d=128, scales=True, mis=0):
    h = ctypes.c_void_p()
    k, v, ks, vs = _bufs(layers, 4)
    if mis:
        ks[0] += mis
    st = L.kvc_create_quantized(ctypes.byref(h), layers, B, Hkv, max_len, d, k, v, ks if scales else None, vs)
    return st, h


def _paged(L, page=128, d=128, pages=4, mpr=2, B=2):
    h = ctypes.c_void_p()
    k, v, ks, vs = _bufs(1, 4)
    st = L.kvc_create_quantized_paged(ctypes.byref(h), 1, B, 2, page, pages, mpr, d, k, v, ks, vs, ctypes.c_void_p(1 << 45))
    return st, h


def _i64(*x):
    a = np.array(x, dtype=np.int64)
    return a, a.ctypes.data_as(I64P)


def _i32(*x):
    a = np.array(x, dtype=np.int32)
    return a, a.ctypes.data_as(I32P)


def test_creation(L):
    for d in (32, 64, 96, 128, 256):
        st, h = _create(L, d=d)
        assert st == 0 and h.value
        L.kvc_destroy(h)
    for kw in (dict(d=16), dict(d=80), dict(d=288), dict(layers=0), dict(B=1025), dict(max_len=0), dict(scales=False),
               dict(mis=8)):
        st, h = _create(L, **kw)
        assert st == ARG and not h.value, kw
    assert L.kvc_create_quantized(None, 1, 1, 1, 8, 64, None, None, None, None) == ARG


def test_plain_creation_refuses_the_type(L):
    h = ctypes.c_void_p()
    k, v = _bufs(1, 2)
    assert L.kvc_create(ctypes.byref(h), 1, 1, 1, 8, 64, _lib.KVC_Q4, k, v) == ARG and not h.value
    assert b"kvc_create_quantized" in L.kvc_last_error()
    assert L.kvc_create_paged(ctypes.byref(h), 1, 1, 1, 128, 2, 2, 64, _lib.KVC_Q4, k, v, ctypes.c_void_p(1 << 45)) == ARG
    assert not h.value


def test_pages_and_rings(L):
    for page, d, want in ((128, 128, 0), (256, 64, 0), (64, 128, ARG), (64, 64, ARG), (20, 96, 0), (0, 96, ARG)):
        st, h = _paged(L, page=page, d=d)
        assert st == want, (page, d)
        if st == 0:
            assert L.kvc_set_window(h, 16, 1) == ARG  # pages do not combine with a ring
            L.kvc_destroy(h)
    for d, max_len, want in ((128, 256, 0), (64, 128, 0), (128, 192, ARG), (64, 100, ARG), (96, 100, 0)):
        st, h = _create(L, d=d, max_len=max_len)
        assert st == 0
        assert L.kvc_set_window(h, 16, 1) == want, (d, max_len)
        L.kvc_destroy(h)


def test_head_scales_do_not_apply(L):
    st, h = _create(L)
    s = np.ones(2, dtype=np.float32)
    fp = ctypes.POINTER(ctypes.c_float)
    assert L.kvc_set_kv_scales(h, 0, s.ctypes.data_as(fp), s.ctypes.data_as(fp)) == ARG
    L.kvc_destroy(h)


@pytest.mark.parametrize("quantized", [True, False])
def test_read_arguments(L, quantized):
    h = ctypes.c_void_p()
    if quantized:
        st, h = _create(L, max_len=128)
    else:
        k, v = _bufs(1, 2)
        st = L.kvc_create(ctypes.byref(h), 1, 2, 2, 128, 128, _lib.KVC_BF16, k, v)
    assert st == 0
    keep, p = _i64(10, 0)
    assert L.kvc_set_lens(h, 0, p) == 0
    out = ctypes.c_void_p(1 << 46)

    def read(first, count, T, k=out, v=out, layer=0):
        (fa, fp), (ca, cp) = _i64(*first), _i32(*count)
        return L.kvc_read(h, layer, fp, cp, T, k, v, None)

    assert read((0, 0), (0, 0), 0) == 0                       # nothing asked: nothing launched
    assert read((99, -5), (0, 0), 4, None, None) == 0         # first is not looked at
    assert read((0, 0), (5, 0), 4) == SHAPE                   # count > T
    assert read((0, 0), (-1, 0), 4) == SHAPE
    assert read((6, 0), (5, 0), 8) == SHAPE                   # past the row's length
    assert read((-1, 0), (2, 0), 8) == SHAPE
    assert read((2 ** 62, 0), (2, 0), 8) == SHAPE
    assert read((0, 0), (1, 1), 8) == SHAPE                   # the second row is empty
    assert read((0, 0), (5, 0), -1) == ARG
    assert read((0, 0), (5, 0), 8, layer=1) == ARG
    assert read((0, 0), (5, 0), 8, k=None) == ARG
    assert read((0, 0), (5, 0), 8, v=ctypes.c_void_p((1 << 46) + 8)) == ARG
    assert L.kvc_read(h, 0, None, None, 8, out, out, None) == ARG
    assert L.kvc_read(None, 0, p, None, 8, out, out, None) == ARG
    L.kvc_destroy(h)


def test_read_of_a_ring_refuses_what_left_it(L):
    st, h = _create(L, max_len=128)
    assert L.kvc_set_window(h, 16, 1) == 0
    keep, p = _i64(300, 100)
    assert L.kvc_set_lens(h, 0, p) == 0
    (fa, fp), (ca, cp) = _i64(171, 0), _i32(4, 4)
    assert L.kvc_read(h, 0, fp, cp, 4, ctypes.c_void_p(1 << 46), ctypes.c_void_p(1 << 46), None) == SHAPE
    L.kvc_destroy(h)


def test_overflow_and_lengths_stay(L):
    st, h = _create(L, max_len=64)
    n, np_ = _i32(65, 1)
    kv = ctypes.c_void_p(1 << 46)
    assert L.kvc_append(h, 0, kv, kv, 65, np_, None) == OVERFLOW
    got = np.zeros(2, dtype=np.int64)
    assert L.kvc_get_lens(h, 0, got.ctypes.data_as(I64P)) == 0 and not got.any()
    L.kvc_destroy(h)
