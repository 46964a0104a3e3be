"""Keys that a query does not see, with infinities and NaN in them, beside it in the tiles of sv_attention_packed."""
import math

import pytest
import torch

from test_gpu_packed_attention import Case

pytestmark = pytest.mark.gpu

# two documents; the second one's first keys share the last tile of the first one's (tiles of two query groups, of
# one, key ranges divided among blocks, few rows)
SHAPES = [([300, 200], [300, 200], 3, 3, 72), ([129, 140], [150, 140], 4, 2, 64), ([260, 9], [513, 130], 40, 40, 128),
          ([130, 60], [1500, 1300], 2, 1, 64), ([40, 17], [9000, 1200], 8, 2, 128), ([70, 33], [1025, 1100], 1, 1, 24),
          ([2, 1], [200, 131], 2, 2, 72), ([3, 1], [5000, 131], 2, 1, 128)]


@pytest.mark.parametrize("poison", [math.nan, math.inf, 900.0])
@pytest.mark.parametrize("lq,lk,hq,hk,d", SHAPES)
def test_capped_scores_do_not_mix(sv, poison, lq, lk, hq, hk, d):
    """Four capped scores share a reciprocal: a hidden key's score leaves the bits of its neighbours alone."""
    c = Case(lq, lk, hq, hk, d, seed=lk[0] + d)
    options = (dict(softcap=5.0), dict(softcap=5.0, mask=1))
    want = [c.run(sv, **opt) for opt in options]
    for opt, w in zip(options, want):
        c.check(w, **opt)
    c.k[lk[0]:] = poison
    for opt, w in zip(options, want):
        assert torch.equal(c.run(sv, **opt)[:lq[0]], w[:lq[0]]), opt
    sv.sv_sync()


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf, 900.0])
@pytest.mark.parametrize("lq,lk,hq,hk,d", SHAPES)
@pytest.mark.parametrize("out", ["f16", "e4m3"])
def test_a_document_keeps_its_bits_beside_another(sv, poison, lq, lk, hq, hk, d, out):
    """Whatever the second document's keys and values are: the first one's rows have the same bits."""
    c = Case(lq, lk, hq, hk, d, seed=lk[0] + d)
    slopes = torch.linspace(0.0, 0.05, hq, device="cuda")
    options = (dict(), dict(mask=1), dict(softcap=5.0), dict(slopes=slopes, mask=1),
               dict(softcap=5.0, slopes=slopes, mask=1, prefix=[3, 3]))
    want = []
    for opt in options:
        want.append(c.run(sv, out=out, **opt))
        c.check(want[-1], out=out, **opt)
    for x in (c.k, c.v):
        x[lk[0]:] = poison
    for opt, w in zip(options, want):
        got = c.run(sv, out=out, **opt)
        assert torch.equal(got[:lq[0]].view(torch.uint8), w[:lq[0]].view(torch.uint8)), opt
    sv.sv_sync()


@pytest.mark.parametrize("poison", [math.nan, math.inf])
@pytest.mark.parametrize("lens,hq,hk,d,key", [([729], 4, 4, 72, 600), ([1500], 2, 1, 64, 1400), ([700, 513], 2, 2, 128, 699)])
def test_rows_of_earlier_tiles_keep_their_bits(sv, poison, lens, hq, hk, d, key):
    """Under the prefix mask an item's products end with the last key that one of its queries sees: queries more than
    256 before a spoiled key have the bits that they have without it."""
    c = Case(lens, lens, hq, hk, d, seed=key)
    want = c.run(sv, mask=1)
    c.check(want, mask=1)
    c.k[key] = poison
    c.v[key] = poison
    got = c.run(sv, mask=1)
    before = key // 256 * 256
    assert torch.equal(got[:before], want[:before])
    assert torch.isfinite(got[before:key]).all() and not torch.isfinite(got[key:lens[0]]).any()
    sv.sv_sync()
