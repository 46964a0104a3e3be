"""sv_rope_plan_init and the argument checks of sv_rope and sv_qk_norm_rope (no GPU)."""
import ctypes
import math

import numpy as np
import pytest

import rope_ref


@pytest.fixture(scope="module")
def vt():
    from vision_transformer_gb300 import build
    build.build()
    import vision_transformer_gb300 as vt
    vt.load()
    return vt


@pytest.mark.parametrize("rot,axes,base,scaling,factor,original", [
    (128, 1, 10000.0, 0, 1.0, 0), (72, 2, 100.0, 0, 1.0, 0), (2, 1, 10000.0, 0, 1.0, 0), (256, 1, 1e6, 1, 4.0, 0),
    (64, 1, 10000.0, 2, 8.0, 0), (128, 1, 500000.0, 3, 8.0, 8192), (36, 1, 10000.0, 3, 1.0, 1)])
def test_plan_frequencies(vt, rot, axes, base, scaling, factor, original):
    """Turns per position to 2^-50 relative: pow and a few operations in 53 bits."""
    p = vt.sv_rope_plan_init(rot, axes, 1, base, scaling, factor, original)
    n = rot // 2 // axes
    f, gain = rope_ref.frequencies(n, base, scaling, factor, original)
    assert (p.rot_dim, p.axes, p.layout, p.pairs) == (rot, axes, 1, n)
    assert abs(p.gain - gain) <= 2.0 ** -24 * gain
    got = np.array([p.turns[i] for i in range(n)], dtype=np.float64) / 2.0 ** 64
    np.testing.assert_allclose(got, f / (2 * math.pi), rtol=2.0 ** -48, atol=2.0 ** -63)


@pytest.mark.parametrize("bad", [
    dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=258), dict(rot_dim=6, axes=2), dict(axes=3), dict(axes=0),
    dict(layout=2), dict(layout=-1), dict(base=0.5), dict(base=math.inf), dict(base=math.nan), dict(scaling=4),
    dict(scaling=1, factor=0.5), dict(scaling=1, factor=math.nan), dict(scaling=2, rot_dim=2, factor=2.0),
    dict(scaling=3, factor=2.0, original_len=0)])
def test_plan_refusals(vt, bad):
    args = dict(rot_dim=64)
    args.update(bad)
    with pytest.raises(vt.SvError) as e:
        vt.sv_rope_plan_init(**args)
    assert e.value.status == vt.SV_ERR_INVALID_ARG


def test_call_refusals(vt):
    """Bad arguments are turned down on the host before any device work."""
    buf = (ctypes.c_uint8 * 4096)()
    p = (ctypes.addressof(buf) + 15) // 16 * 16
    plan = vt.sv_rope_plan_init(64)
    lib, bad = vt.load(), vt.SV_ERR_INVALID_ARG

    def rope(x=p, y=p, pos=p, plan=plan, rows=1, heads=1, d=64, xs=0, ys=0):
        return lib.sv_rope(x, y, pos, plan, rows, heads, d, xs, ys, None)

    def qk(q=p, k=p, qo=p, ko=p, qg=p, kg=p, norm=0, eps=1e-6, pos=p, plan=plan, rows=1, hq=1, hk=1, d=64, qs=0, ks=0,
           qos=0, kos=0):
        return lib.sv_qk_norm_rope(q, k, qo, ko, qg, kg, norm, eps, pos, plan, rows, hq, hk, d, qs, ks, qos, kos, None)

    for kw in (dict(x=None), dict(y=None), dict(pos=None), dict(plan=None), dict(rows=-1), dict(heads=0), dict(d=0),
               dict(d=60), dict(d=264), dict(d=56), dict(xs=56), dict(ys=68), dict(x=p + 2), dict(y=p + 8),
               dict(pos=p + 2), dict(heads=2, xs=64), dict(xs=64, ys=72)):
        assert rope(**kw) == bad, kw
    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(norm=2), dict(eps=-1.0),
               dict(eps=math.nan), dict(hq=0), dict(hk=0), dict(qg=p + 8), dict(kg=p + 4), dict(qs=8), dict(kos=68),
               dict(pos=None), dict(rows=-1), dict(qs=72), dict(kos=72)):
        assert qk(**kw) == bad, kw
    broken = vt.sv_rope_plan_init(64)
    broken.pairs = 64
    assert rope(plan=broken) == bad and b"sv_rope_plan_init" in lib.sv_last_error()
    # no rows is no work
    assert rope(rows=0) == vt.SV_OK and qk(rows=0) == vt.SV_OK


def test_too_many_heads(vt):
    buf = (ctypes.c_uint8 * 4096)()
    p = (ctypes.addressof(buf) + 15) // 16 * 16
    plan = vt.sv_rope_plan_init(8)
    lib = vt.load()
    assert lib.sv_rope(p, p, p, plan, 1, 2 ** 20 + 1, 8, 0, 0, None) == vt.SV_ERR_INVALID_ARG
    for hq, hk in ((2 ** 20 + 1, 1), (1, 2 ** 20 + 1)):
        assert lib.sv_qk_norm_rope(p, p, p, p, None, None, 0, 1e-6, p, plan, 1, hq, hk, 8, 0, 0, 0, 0,
                                   None) == vt.SV_ERR_INVALID_ARG
