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


def decode(lib, out=P, q=P, kp=P, vp=P, nb=10, tables=P, mb=4, lens=P, max_len=64, S=2, hq=8, hkv=4,
           d=128, bs=16, scale=1.0, part=-1, ws=NULL, wsb=0, dt=1):
    return lib.pa_decode_int4(out, q, kp, vp, nb, tables, mb, lens, max_len, S, hq, hkv, d, bs,
                              ctypes.c_float(scale), part, ws, wsb, dt, NULL)


def test_decode_refusals(lib):
    for kw in (dict(out=NULL), dict(q=NULL), dict(kp=NULL), dict(vp=NULL), dict(tables=NULL),
               dict(lens=NULL), dict(out=ODD), dict(q=ODD), dict(kp=ODD), dict(nb=0), dict(mb=-1),
               dict(max_len=-1), dict(S=-1), dict(hq=6), dict(hkv=0), dict(dt=5),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(part=-2), dict(part=24),
               dict(part=8), dict(S=70000)):
        assert decode(lib, **kw) == INVALID, kw
    for kw in (dict(d=96), dict(d=256), dict(bs=24), dict(bs=64), dict(hq=36)):
        assert decode(lib, **kw) == UNSUPPORTED, kw
    assert lib.pa_decode_int4_workspace_size(2, 8, 4, 128, 16, 64, -1, 1) == 0
    assert lib.pa_decode_int4_workspace_size(2, 8, 4, 128, 16, 64, 16, 1) > 2 * 8 * 4 * 128 * 4
    assert lib.pa_decode_int4_workspace_size(2, 8, 4, 96, 16, 64, 16, 1) == 0


def rope(lib, qo=P, qos=512, q=P, qs=512, k=P, ks=256, v=P, vs=256, qw=P, kw=P, eps=1e-6, cs=P,
         npos=10, rot=128, inter=0, pos=P, slots=P, T=3, kp=P, vp=P, nb=4, hq=4, hkv=2, d=128,
         bs=16, fmt=0, ksc=1.0, vsc=1.0, dt=1):
    f = ctypes.c_float
    return lib.pa_qk_norm_rope(qo, qos, q, qs, k, ks, v, vs, qw, kw, f(eps), cs, npos, rot, inter,
                               pos, slots, T, kp, vp, nb, hq, hkv, d, bs, fmt, f(ksc), f(vsc), dt,
                               NULL)


def test_norm_rope_refusals(lib):
    for name in ("qo", "q", "k", "v", "qw", "kw", "cs", "kp", "vp"):
        assert rope(lib, **{name: NULL}) == INVALID, name
        assert rope(lib, **{name: ODD}) == INVALID, name
    for kw in (dict(pos=NULL), dict(slots=NULL), dict(T=-1), dict(nb=0), dict(hq=3), dict(hkv=0),
               dict(hq=0), dict(npos=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(qs=504), dict(qos=504), dict(ks=248), dict(vs=248),
               dict(qs=516), dict(qos=516), dict(ks=260), dict(vs=260), dict(dt=2), dict(fmt=3),
               dict(fmt=-1), dict(fmt=1, ksc=0.0), dict(fmt=1, vsc=-1.0),
               dict(fmt=1, ksc=float("inf")), dict(fmt=1, vsc=float("nan"))):
        assert rope(lib, **kw) == INVALID, kw
    for kw in (dict(d=96, rot=96), dict(bs=8), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144)):
        assert rope(lib, **kw) == UNSUPPORTED, kw
    assert rope(lib, T=0) == 0


def test_decode_and_norm_rope_wrappers_refuse(lib):
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    pool = torch.zeros(api.int4_pool_shape(4, 2, 16, 128), dtype=torch.uint8)
    tables, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for args in ((q[:2], q, pool, pool, tables, lens), (q.half(), q, pool, pool, tables, lens),
                 (q, q, pool[..., :-1], pool[..., :-1], tables, lens),
                 (q, q, pool, pool, tables[:2], lens), (q, q, pool, pool, tables, lens[:2]),
                 (q, q, pool[0], pool[0], tables, lens), (q, q, pool, pool, tables, lens)):
        with pytest.raises(ValueError):
            api.decode_int4(*args, 16, 1.0)
    with pytest.raises(TypeError):
        api.decode_int4(q.float(), q.float(), pool, pool, tables, lens, 16, 1.0)

    k, w, cs = torch.zeros(3, 2, 128, dtype=torch.bfloat16), q[0, 0], torch.zeros(9, 128)
    n = torch.zeros(3, dtype=torch.int64)
    wide = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    for change in ({0: q[:2]}, {2: k[:2]}, {3: k[:, :1]}, {4: w[:64]}, {5: w[:64]}, {8: n[:2]},
                   {9: n[:2]}, {10: wide[..., :64], 11: wide[..., :64]}, {11: wide[:3]},
                   {10: wide.to(torch.uint8), 11: wide.to(torch.uint8)}, {}):
        args = [q, q, k, k, w, w, 1e-6, cs, n, n, wide, wide]
        for i, t in change.items():
            args[i] = t
        with pytest.raises(ValueError):
            api.qk_norm_rope(*args)
    for change in ({2: k.half()}, {4: w.float()}, {10: wide.float(), 11: wide.float()}, {10: pool}):
        args = [q, q, k, k, w, w, 1e-6, cs, n, n, wide, wide]
        for i, t in change.items():
            args[i] = t
        with pytest.raises(TypeError):
            api.qk_norm_rope(*args)
