"""sv_attention_packed with caps of any size.

Tolerance: as packed_ref.bound without its term for the cap (2^-21 of the cap, which says nothing for large ones), and
2^-18 of the score more: 64 2^-24 of its terms, as if the head were 64 wider.
"""
import pytest
import torch

import packed_ref
from test_gpu_packed_attention import Case

pytestmark = pytest.mark.gpu


def _check(c, o, out, softcap, **opt):
    got = (o.view(torch.float8_e4m3fn).double() / 16) if out == "e4m3" else o.double()
    for _, a, lq, q, k, v in c.docs():
        ref, av, terms = packed_ref.document(q, k, v, softcap=softcap, **opt)
        tol = packed_ref.bound(ref, av, terms, k.shape[0], float(v.abs().max()), c.d + 64, 0.0, out == "e4m3")
        err = (got[a:a + lq].reshape(ref.shape) - ref).abs()
        assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("cap,scale_q", [(256.0, 1.0), (256.0, 60.0), (300.0, 200.0), (1e4, 1.0), (1e4, 3000.0), (1e6, 1.0),
                                         (1e6, 30.0), (1e30, 2.0), (3e38, 2.0)])
@pytest.mark.parametrize("lq,lk,hq,hk,d", [([300, 70], [300, 70], 4, 2, 64), ([130], [1500], 2, 2, 128),
                                           ([40], [9000], 8, 2, 128), ([1, 2], [700, 5000], 4, 4, 72)])
@pytest.mark.parametrize("out", ["f16", "e4m3"])
def test_large_caps(sv, cap, scale_q, lq, lk, hq, hk, d, out):
    """Scores far below the cap, where they all but stay, near it and beyond it."""
    c = Case(lq, lk, hq, hk, d, seed=d, scale_q=scale_q)
    slopes = torch.linspace(0.0, 0.5, hq, device="cuda")
    for opt in (dict(), dict(mask=1), dict(mask=1, slopes=slopes)):
        o = c.run(sv, out=out, softcap=cap, **opt)
        _check(c, o, out, cap, **opt)
        assert torch.equal(o.view(torch.uint8), c.run(sv, out=out, softcap=cap, workspace=c.ws, **opt).view(torch.uint8))
    sv.sv_sync()


@pytest.mark.parametrize("cap", [1e-39, 1e-30, 1e-3])
@pytest.mark.parametrize("lq,lk", [([300, 70], [300, 70]), ([130], [1500]), ([1, 2], [700, 5000])])
def test_small_caps(sv, cap, lq, lk):
    """Scores that vanish against any difference: every key counts the same, products of 0 among them."""
    c = Case(lq, lk, 2, 1, 64, seed=1)
    c.q[::2] = 0
    o = c.run(sv, softcap=cap)
    # (a score of +-cap moves a probability by at most 2 cap of itself)
    for _, a, n, q, k, v in c.docs():
        ref = v.double().mean(0).repeat(n, 2, 1)
        tol = packed_ref.bound(ref, v.double().abs().mean(0).repeat(n, 2, 1), torch.zeros_like(ref[..., :1]), v.shape[0],
                               float(v.abs().max()), 64) + 2.1 * cap * float(v.abs().max())
        assert ((o[a:a + n].reshape(ref.shape).double() - ref).abs() <= tol).all()
    sv.sv_sync()
