"""Refusals of the 4-bit cache's entry points: no device call is needed, so
these run without a GPU (pointers are never followed)."""
import ctypes

import pytest
import torch

from paged_kv_cache_64_gb300 import _lib, api

P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
NULL = ctypes.c_void_p(0)
INVALID, UNSUPPORTED = 1, 3


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_64_gb300 import build
    build.build()
    return _lib.load()


def write(lib, k=P, v=P, slots=P, tokens=3, kp=P, vp=P, nb=4, hkv=2, d=128, bs=16, ko=NULL, vo=NULL,
          dt=1):
    return lib.pa_cache_write_int4(k, v, slots, tokens, kp, vp, nb, hkv, d, bs, ko, vo, dt, NULL)


def read(lib, ko=P, vo=P, slots=P, tokens=3, kp=P, vp=P, nb=4, hkv=2, d=128, bs=16, dt=1):
    return lib.pa_cache_read_int4(ko, vo, slots, tokens, kp, vp, nb, hkv, d, bs, dt, NULL)


def test_record_bytes(lib):
    assert [lib.pa_int4_record_bytes(d, b) for d in (64, 128) for b in (16, 32)] == [
        576, 1152, 1088, 2176]
    assert lib.pa_int4_record_bytes(96, 16) == 0 and lib.pa_int4_record_bytes(128, 8) == 0
    assert api.int4_pool_shape(7, 2, 16, 128) == (7, 2, 1088)
    with pytest.raises(ValueError):
        api.int4_pool_shape(7, 2, 24, 128)


@pytest.mark.parametrize("call", [write, read])
def test_refusals(lib, call):
    for kw in (dict(tokens=-1), dict(nb=0), dict(hkv=0), dict(dt=2), dict(slots=NULL),
               dict(kp=NULL), dict(vp=NULL), dict(kp=ODD), dict(vp=ODD),
               dict(tokens=1 << 30, hkv=2)):
        assert call(lib, **kw) == INVALID, kw
    for kw in (dict(d=96), dict(d=256), dict(bs=8), dict(bs=64), dict(bs=0)):
        assert call(lib, **kw) == UNSUPPORTED, kw
    assert call(lib, tokens=0) == 0  # nothing to do, nothing launched


def test_refusals_of_the_rows(lib):
    for kw in (dict(k=NULL), dict(v=NULL), dict(k=ODD), dict(v=ODD), dict(ko=P), dict(vo=P),
               dict(ko=ODD, vo=P), dict(ko=P, vo=ODD)):
        assert write(lib, **kw) == INVALID, kw
    for kw in (dict(ko=NULL), dict(vo=NULL), dict(ko=ODD), dict(vo=ODD)):
        assert read(lib, **kw) == INVALID, kw


def test_wrappers_refuse_bad_shapes_and_host_tensors(lib):
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    pool = torch.zeros(api.int4_pool_shape(4, 2, 16, 128), dtype=torch.uint8)
    slots = torch.zeros(3, dtype=torch.int64)
    for args, kw in (
            ((k, k[:2], slots, pool, pool), {}),
            ((k, k.half(), slots, pool, pool), {}),
            ((k, k, slots[:2], pool, pool), {}),
            ((k, k, slots, pool[..., :-16], pool[..., :-16]), {}),
            ((k, k, slots, pool[:, :1], pool[:, :1]), {}),
            ((k, k, slots, pool, pool[:3]), {}),
            ((k, k, slots, pool, pool), dict(k_out=k)),
            ((k, k, slots, pool, pool), dict(k_out=k, v_out=k.half())),
            ((k, k, slots, pool, pool), {})):  # the last: host tensors
        with pytest.raises(ValueError):
            api.cache_write_int4(*args, **kw)
    with pytest.raises(TypeError):
        api.cache_write_int4(k, k, slots, pool.to(torch.int8), pool)
    for args in ((k, k[:2], slots, pool, pool), (k, k, slots[:2], pool, pool),
                 (k, k, slots, pool[..., :-4], pool[..., :-4]), (k, k, slots, pool, pool)):
        with pytest.raises(ValueError):
            api.cache_read_int4(*args)
