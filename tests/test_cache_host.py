"""Argument checks of sv_cache_write, sv_cache_read and sv_attention_cached (no GPU)."""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def vt():
    from vision_transformer_gb300 import build
    build.build()
    import vision_transformer_gb300 as vt
    vt.load()
    return vt


@pytest.fixture
def p():
    buf = (ctypes.c_uint8 * 4096)()
    yield (ctypes.addressof(buf) + 127) // 128 * 128
    del buf


def _cache(vt, p, pages=None, n=4, page=16, heads=2, dim=64, dtype=1):
    return vt.sv_cache(p if pages is None else pages, n, page, heads, dim, dtype)


def _batch(vt, p, count=2, table=None, stride=3, lengths=None, prefix_pages=None, prefix=0):
    return vt.sv_cache_batch(count, p if table is None else table, stride, p if lengths is None else lengths, prefix_pages,
                             prefix)


@pytest.mark.parametrize("page,heads,dim,dtype,want", [(16, 1, 8, 1, 384), (64, 8, 128, 1, 2 * 8 * 64 * 129),
                                                       (32, 16, 72, 0, 2 * 16 * 32 * 145), (16, 3, 72, 1, 7040)])
def test_page_bytes(vt, page, heads, dim, dtype, want):
    assert vt.sv_cache_page_bytes(page, heads, dim, dtype) == want


@pytest.mark.parametrize("page,heads,dim,dtype", [(8, 1, 64, 1), (48, 1, 64, 1), (512, 1, 64, 1), (16, 0, 64, 1),
                                                  (16, 1, 60, 1), (16, 1, 136, 1), (16, 1, 64, 2), (16, 1, 0, 0)])
def test_pages_that_no_cache_has(vt, page, heads, dim, dtype):
    assert vt.sv_cache_page_bytes(page, heads, dim, dtype) == 0


@pytest.mark.parametrize("fn", ["sv_cache_write", "sv_cache_read"])
def test_refusals_of_write_and_read(vt, p, fn):
    """Bad arguments are turned down on the host before any device work."""
    call = getattr(vt.load(), fn)
    inv, uns = vt.SV_ERR_INVALID_ARG, vt.SV_ERR_UNSUPPORTED

    def go(cache=(), batch=(), k=p, v=p, off=p, total=4, ks=0, vs=0):
        c = _cache(vt, p, **dict(cache)) if cache is not None else None
        b = _batch(vt, p, **dict(batch)) if batch is not None else None
        return call(c, b, k, v, off, total, ks, vs, None)

    for kw in (dict(cache=None), dict(batch=None), dict(cache=dict(n=0)), dict(cache=dict(heads=0)),
               dict(cache=dict(dtype=2)), dict(cache=dict(pages=0)), dict(cache=dict(pages=p + 8)),
               dict(batch=dict(count=0)), dict(batch=dict(stride=-1)), dict(batch=dict(prefix=-1)),
               dict(batch=dict(table=0)), dict(batch=dict(table=p + 2)), dict(batch=dict(lengths=0)),
               dict(batch=dict(lengths=p + 1)), dict(batch=dict(prefix=5)),
               dict(batch=dict(prefix=5, prefix_pages=p + 2)), dict(total=-1), dict(k=None), dict(v=None), dict(k=p + 8),
               dict(v=p + 2), dict(off=p + 2), dict(off=None, total=5), dict(ks=120), dict(vs=132)):
        assert go(**kw) == inv, kw
    for kw in (dict(cache=dict(page=8)), dict(cache=dict(page=24)), dict(cache=dict(dim=68)), dict(cache=dict(dim=136)),
               dict(cache=dict(heads=65537)), dict(total=2 ** 31 - 1), dict(batch=dict(stride=2 ** 27)),
               dict(batch=dict(prefix=2 ** 31 - 1, prefix_pages=p)), dict(cache=dict(heads=64, dim=8), total=2 ** 27)):
        assert go(**kw) == uns, kw
    assert go(total=0) == vt.SV_OK


def test_refusals_of_attention(vt, p):
    lib, inv, uns = vt.load(), vt.SV_ERR_INVALID_ARG, vt.SV_ERR_UNSUPPORTED
    opt = vt.sv_attention_options

    def go(cache=(), batch=(), q=p, o=p, off=p, total=4, heads=4, qs=0, os=0, options=None, out=0, ws=p, size=1 << 30):
        c = _cache(vt, p, **dict(cache)) if cache is not None else None
        b = _batch(vt, p, **dict(batch)) if batch is not None else None
        return lib.sv_attention_cached(c, b, q, o, off, total, heads, qs, os, options, out, ws, size, None)

    for kw in (dict(cache=None), dict(batch=None), dict(q=None), dict(o=None), dict(q=p + 8), dict(o=p + 2),
               dict(heads=0), dict(heads=3), dict(heads=-2), dict(total=-1), dict(off=None, total=3), dict(off=p + 2),
               dict(qs=248), dict(os=260), dict(out=2), dict(ws=None), dict(ws=p + 8), dict(size=64),
               dict(options=opt(mask=2)), dict(options=opt(softcap=-1.0)), dict(options=opt(softcap=math.inf)),
               dict(options=opt(scale=math.nan)), dict(batch=dict(lengths=0)), dict(cache=dict(pages=0))):
        assert go(**kw) == inv, kw
    for kw in (dict(options=opt(prefix=p)), dict(options=opt(slopes=p)), dict(heads=130), dict(cache=dict(dim=12)),
               dict(cache=dict(page=20)), dict(batch=dict(count=2 ** 24 + 1)), dict(total=2 ** 25)):
        assert go(**kw) == uns, kw
    assert go(total=0) == vt.SV_OK
    assert go(total=0, ws=None, size=0) == vt.SV_OK


def test_workspace_does_not_depend_on_lengths(vt, p):
    def size(total, heads=32, prefix=0, stride=3):
        return vt.sv_attention_cached_workspace(_cache(vt, p, heads=8, dim=128),
                                                _batch(vt, p, count=16, stride=stride, prefix=prefix,
                                                       prefix_pages=p if prefix else None), total, heads)

    assert 0 < size(16) <= 40 << 20 and size(16) == size(16, stride=10000)
    assert size(0) == 0
    assert size(0, stride=10 ** 6) == 0
    # 32 rows of a head and sequence on average and no more; else tiles of 128 rows
    assert 0 < size(128) <= 40 << 20
    assert 4096 * 32 * 130 * 4 < size(4096) <= 11 * 2 ** 20 + (4096 + 16 * 32) * 32 * 130 * 4
    for prefix in (1, 1000, 10 ** 6):
        assert 0 < size(1024, prefix=prefix) <= (32 << 20) + (2 * 1024 * 32 + 16 * 8 * 128 + 8 * 256) * 130 * 4
