"""Refusals of the latent cache's entry points: no device call is needed, so
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


def rope(lib, qo=P, qot=1024, qoh=64, q=P, qt=1024, qh=64, x=P, xs=576, w=P, eps=1e-6, cs=P, npos=10,
         pos=P, slots=P, tokens=3, rows=NULL, pool=P, nb=4, heads=16, rank=512, bs=16, dt=1):
    return lib.pa_latent_norm_rope(qo, qot, qoh, q, qt, qh, x, xs, w, eps, cs, npos, 0, pos, slots,
                                   tokens, rows, pool, nb, heads, rank, bs, dt, NULL)


def read(lib, rows=P, slots=P, tokens=3, pool=P, nb=4, rank=512, bs=16, dt=1):
    return lib.pa_cache_read_latent(rows, slots, tokens, pool, nb, rank, bs, dt, NULL)


def decode(lib, out=P, q=P, pool=P, nb=4, tables=P, mb=2, lens=P, max_len=30, S=2, heads=16, rank=512,
           bs=16, scale=0.1, ws=NULL, wb=0, dt=1):
    return lib.pa_decode_latent(out, q, pool, nb, tables, mb, lens, max_len, S, heads, rank, bs, scale,
                                ws, wb, dt, NULL)


def prefill(lib, out=P, q=P, qt=3264, qh=192, k=P, kt=4096, kh=256, v=P, vt=4096, vh=256, pe=P,
            pt=576, qs=P, ks=P, S=2, tq=10, tk=12, mq=5, heads=16, scale=0.1, causal=1, dt=1):
    return lib.pa_prefill_latent(out, q, qt, qh, k, kt, kh, v, vt, vh, pe, pt, qs, ks, S, tq, tk, mq,
                                 heads, scale, causal, dt, NULL)


def test_rope_refusals(lib):
    for kw in (dict(tokens=-1), dict(nb=0), dict(heads=0), dict(npos=0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(dt=2), dict(qot=56), dict(qoh=60), dict(qt=1028), dict(qh=0),
               dict(xs=568), dict(xs=577), dict(heads=1 << 23), dict(qo=NULL), dict(q=ODD), dict(x=ODD),
               dict(w=ODD), dict(cs=ODD), dict(pool=ODD), dict(rows=ODD), dict(pos=NULL),
               dict(slots=NULL)):
        assert rope(lib, **kw) == INVALID, kw
    for kw in (dict(rank=128), dict(rank=576), dict(bs=8), dict(bs=128)):
        assert rope(lib, **kw) == UNSUPPORTED, kw
    assert rope(lib, tokens=0) == 0


def test_read_refusals(lib):
    for kw in (dict(tokens=-1), dict(nb=0), dict(dt=5), dict(rows=NULL), dict(rows=ODD), dict(pool=ODD),
               dict(slots=NULL)):
        assert read(lib, **kw) == INVALID, kw
    for kw in (dict(rank=64), dict(bs=48)):
        assert read(lib, **kw) == UNSUPPORTED, kw
    assert read(lib, tokens=0) == 0


def test_decode_refusals(lib):
    for kw in (dict(S=-1), dict(S=65536), dict(nb=0), dict(mb=0), dict(max_len=-1), dict(heads=0),
               dict(heads=1025), dict(scale=float("inf")), dict(dt=2), dict(out=NULL), dict(q=ODD),
               dict(pool=ODD), dict(tables=NULL), dict(lens=NULL), dict(nb=1 << 27),
               dict(mb=1 << 27), dict(mb=1 << 21, max_len=(1 << 24) + 1),
               dict(S=65535, max_len=1 << 24, mb=1 << 20)):
        assert decode(lib, **kw) == INVALID, kw
    for kw in (dict(rank=128), dict(bs=8)):
        assert decode(lib, **kw) == UNSUPPORTED, kw
    assert decode(lib, S=0) == 0


def test_prefill_refusals(lib):
    for kw in (dict(S=-1), dict(S=65536), dict(tq=-1), dict(tk=-1), dict(mq=-1), dict(heads=0),
               dict(heads=1025), dict(scale=float("nan")), dict(dt=3), dict(qt=184), dict(qh=190),
               dict(kt=120), dict(kh=129), dict(vh=64), dict(pt=32), dict(vt=1 << 39), dict(out=NULL),
               dict(q=ODD), dict(k=NULL), dict(v=ODD), dict(pe=ODD), dict(qs=NULL), dict(ks=NULL),
               dict(tk=(1 << 24) + 1)):
        assert prefill(lib, **kw) == INVALID, kw
    for kw in (dict(S=0), dict(tq=0), dict(mq=0)):
        assert prefill(lib, **kw) == 0, kw


def test_wrappers_refuse_bad_shapes_types_and_host_tensors(lib):
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)
    i64 = torch.zeros(3, dtype=torch.int64)
    good = dict(q_out=h(3, 4, 64), q=h(3, 4, 64), latent=h(3, 320), weight=h(256), eps=1e-6,
                cos_sin=torch.zeros(9, 64), positions=i64, slot_mapping=i64, pool=h(2, 16, 320))
    for kw, err in ((dict(q=h(3, 4, 32)), ValueError), (dict(q_out=h(3, 5, 64)), ValueError),
                    (dict(latent=h(3, 576)), ValueError), (dict(latent=h(4, 320)), ValueError),
                    (dict(weight=h(512)), ValueError), (dict(positions=i64[:2]), ValueError),
                    (dict(cos_sin=torch.zeros(9, 32)), ValueError), (dict(rows_out=h(3, 256)), ValueError),
                    (dict(pool=h(2, 320)), ValueError), (dict(pool=torch.zeros(2, 16, 320)), TypeError),
                    (dict(weight=torch.zeros(256)), TypeError), ({}, ValueError)):
        with pytest.raises(err):
            api.latent_norm_rope(**{**good, **kw})
    with pytest.raises(ValueError):
        api.cache_read_latent(h(3, 320), i64, h(2, 16, 320))
    with pytest.raises(ValueError):
        api.cache_read_latent(h(3, 256), i64, h(2, 16, 320))
    lens = torch.zeros(2, dtype=torch.int32)
    good = dict(out=h(2, 4, 256), q=h(2, 4, 320), pool=h(2, 16, 320), block_tables=lens[:, None],
                seq_lens=lens, max_seq_len=3, scale=0.1)
    for kw, err in ((dict(out=h(2, 4, 320)), ValueError), (dict(q=h(2, 4, 576)), ValueError),
                    (dict(seq_lens=lens[:1]), ValueError), (dict(block_tables=lens), ValueError),
                    (dict(pool=h(2, 16, 320).bfloat16()), TypeError), ({}, ValueError)):
        with pytest.raises(err):
            api.decode_latent(**{**good, **kw})
    good = dict(out=h(5, 4, 128), q=h(5, 4, 192), k=h(6, 4, 128), v=h(6, 4, 128), k_pe=h(6, 64),
                q_starts=lens, k_starts=lens, max_q_len=5, scale=0.1)
    for kw, err in ((dict(q=h(5, 4, 128)), ValueError), (dict(k=h(6, 3, 128)), ValueError),
                    (dict(v=h(5, 4, 128)), ValueError), (dict(k_pe=h(5, 64)), ValueError),
                    (dict(out=h(5, 4, 192)), ValueError), (dict(k_starts=lens[:1]), ValueError),
                    (dict(v=torch.zeros(6, 4, 128)), TypeError), ({}, ValueError)):
        with pytest.raises(err):
            api.prefill_latent(**{**good, **kw})


def test_steps_of_strided_tensors():
    t = torch.zeros(4, 6, 256, dtype=torch.float16)
    assert api._steps(t[..., :128], "k") == (1536, 256)
    assert api._steps(t[:1, :1, :128], "k") == (128, 128)
    assert api._steps(t.transpose(0, 1)[..., :64], "k") == (256, 1536)
    for bad in (t[..., ::2], t[:, :1].expand(4, 6, 256), torch.zeros(4, 6, 65)[..., :64]):
        with pytest.raises(ValueError):
            api._steps(bad, "k")
