"""Argument checks of sv_attention_packed (no GPU)."""
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


def test_refusals(vt):
    """Bad arguments are turned down on the host before any device work."""
    buf = (ctypes.c_uint8 * 4096)()
    p = (ctypes.addressof(buf) + 15) // 16 * 16
    lib, inv, uns = vt.load(), vt.SV_ERR_INVALID_ARG, vt.SV_ERR_UNSUPPORTED

    def call(q=p, k=p, v=p, o=p, qf=p, kf=p, docs=2, tq=4, tk=4, hq=2, hk=1, d=64, qs=0, ks=0, vs=0, os=0, opt=None,
             out=0, ws=None, wb=0):
        return lib.sv_attention_packed(q, k, v, o, qf, kf, docs, tq, tk, hq, hk, d, qs, ks, vs, os, opt, out, ws, wb,
                                       None)

    opt = vt.sv_attention_options
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(docs=0), dict(tq=-1), dict(tk=-1),
               dict(hq=0), dict(hk=0), dict(hq=3, hk=2), dict(out=2), dict(q=p + 8), dict(k=p + 2), dict(v=p + 4),
               dict(o=p + 8), dict(qf=p + 2), dict(kf=p + 1), dict(qs=120), dict(ks=56), dict(vs=68), dict(os=132),
               dict(qf=None, tq=5), dict(kf=None, tk=3), dict(ws=p, wb=8), dict(ws=p + 8, wb=1 << 30),
               dict(opt=opt(mask=2)), dict(opt=opt(softcap=-1.0)), dict(opt=opt(softcap=math.inf)),
               dict(opt=opt(softcap=math.nan)), dict(opt=opt(scale=math.nan)), dict(opt=opt(prefix=p + 2)),
               dict(opt=opt(slopes=p + 1))):
        assert call(**kw) == inv, kw
    for kw in (dict(d=60), dict(d=0), dict(d=136), dict(d=256), dict(hq=65, hk=1)):
        assert call(**kw) == uns, kw
    # no queries is no work
    assert call(tq=0) == vt.SV_OK


@pytest.mark.parametrize("docs,tq,tk,hq,hk,d", [(1, 1, 1, 1, 1, 8), (64, 64, 1 << 20, 32, 8, 128),
                                                 (1, 1 << 20, 1 << 20, 64, 1, 128), (5000, 0, 0, 16, 16, 72)])
def test_workspace_is_bounded(vt, docs, tq, tk, hq, hk, d):
    """The workspace does not grow with the sequences."""
    n = vt.sv_attention_packed_workspace(docs, tq, tk, hq, hk, d)
    assert 0 < n <= 64 << 20


def test_sizes_too_large_for_one_call(vt):
    """Turned down before any device work, whatever the pointers."""
    buf = (ctypes.c_uint8 * 4096)()
    p = (ctypes.addressof(buf) + 15) // 16 * 16
    lib = vt.load()
    most = 2 ** 31 - 1 - 4096
    for docs, tq, tk, hq, hk in ((1, most + 1, 4, 1, 1), (1, 4, most + 1, 1, 1), (2 ** 24 + 1, 4, 4, 1, 1),
                                 (1, most, 4, 1024, 1024), (2 ** 24, 4, 4, 128, 64)):
        assert lib.sv_attention_packed(p, p, p, p, p, p, docs, tq, tk, hq, hk, 8, 0, 0, 0, 0, None, 0, None, 0,
                                       None) == vt.SV_ERR_UNSUPPORTED, (docs, tq, tk, hq, hk)


@pytest.mark.parametrize("tq,hq,hk", [(64, 16, 16), (4096, 32, 8)])
def test_workspace_of_smaller_key_totals(vt, tq, hq, hk):
    """The workspace does not shrink as total_k grows."""
    sizes = [vt.sv_attention_packed_workspace(4, tq, tk, hq, hk, 72) for tk in (0, 1, 1024, 1025, 5000, 10 ** 5, 10 ** 9)]
    assert sizes == sorted(sizes)
