"""Keys that a query does not see, with infinities and NaN in them, beside it in the tiles of sv_attention_packed."""
import math
import time

import pytest
import torch

import packed_ref
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


def _but_the_last_row(c, o, **opt):
    """The rows of the first document but its last query against the formulas."""
    n, _, lq, q, k, v = next(c.docs())
    ref, av, terms = packed_ref.document(q[:-1], k[:-1], v[:-1], **opt)
    tol = packed_ref.bound(ref, av, terms, k.shape[0], float(v[:-1].abs().max()), c.d)
    got = o[:lq].reshape(lq, c.hq, c.d).double()
    assert torch.isfinite(got[:-1]).all() and ((got[:-1] - ref).abs() <= tol).all()
    assert not torch.isfinite(got[-1]).any()
    assert torch.isfinite(o[lq:]).all()


@pytest.mark.parametrize("poison", [math.nan, math.inf])
@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("lq,hq,hk", [(32, 1, 1), (3, 2, 1), (5, 2, 2)])
def test_a_spoiled_key_at_the_end_of_a_long_range(sv, poison, workspace, lq, hq, hk):
    """The last query sees it, the others do not: their rows are computed again, in a time that the waits of the items
    behind them allow."""
    rest = [lq] * 400
    c = Case([lq] + rest, [150000] + rest, hq, hk, 128, seed=lq)
    c.k[149999] = poison
    c.v[149999] = poison
    o = c.run(sv, mask=1, workspace=workspace)
    sv.sv_sync()
    _but_the_last_row(c, o, mask=1)


def test_rows_computed_again_for_longer_than_a_wait_may_last(sv):
    """The waits of the other warps count the progress of rows that are computed again."""
    n = 600000
    rest = [32] * 400
    c = Case([32] + rest, [n] + rest, 1, 1, 128, seed=1)
    c.v[n - 1] = math.nan
    torch.cuda.synchronize()
    start = time.perf_counter()
    o = c.run(sv, mask=1, workspace=False)
    sv.sv_sync()
    print("%.2f s" % (time.perf_counter() - start))
    _but_the_last_row(c, o, mask=1)


@pytest.mark.parametrize("lq,lk,hq,hk,d", [([300], [300], 3, 3, 72), ([1500], [1500], 2, 1, 64), ([40], [9000], 8, 2, 128),
                                           ([6], [9000], 2, 1, 128), ([9], [4000], 4, 4, 72)])
@pytest.mark.parametrize("out", ["f16", "e4m3"])
def test_rows_beside_a_spoiled_key(sv, lq, lk, hq, hk, d, out):
    """A key that only the last queries see, in either output type: those before it as if it were not there."""
    c = Case(lq, lk, hq, hk, d, seed=d)
    slopes = torch.linspace(0.0, 0.05, hq, device="cuda")
    for opt in (dict(), dict(softcap=5.0), dict(slopes=slopes)):
        want = c.run(sv, out=out, mask=1, **opt)
        c.check(want, out=out, mask=1, **opt)
        k, v = c.k.clone(), c.v.clone()
        c.k[-3] = math.nan
        c.v[-3] = math.inf
        got = c.run(sv, out=out, mask=1, **opt)
        spoiled, c.k, c.v = got.clone(), k, v
        # (the last three rows, which see it, are put right to check the others)
        got[-3:] = want[-3:]
        c.check(got, out=out, mask=1, **opt)
        last = spoiled[-3:] if out == "f16" else spoiled[-3:].view(torch.float8_e4m3fn).float()
        assert torch.isnan(last).all()
    sv.sv_sync()


@pytest.mark.parametrize("poison", [math.nan, math.inf])
@pytest.mark.parametrize("hq,hk,d", [(2, 2, 72), (2, 1, 64), (4, 4, 72), (1, 1, 128)])
def test_few_rows_read_no_key_behind_their_block(sv, poison, hq, hk, d):
    """One document of more rows than a block among many single queries: blocks whose queries do not see a spoiled key
    (8 rows each) have the bits that they have without it."""
    lq, lk = [40] + [1] * 20, [30000] + [50] * 20
    c = Case(lq, lk, hq, hk, d, seed=d + hq)
    for workspace in (True, False):
        want = c.run(sv, mask=1, workspace=workspace)
        c.check(want, mask=1)
        k, v = c.k.clone(), c.v.clone()
        c.k[30000 - 5] = poison
        c.v[30000 - 5] = poison
        got = c.run(sv, mask=1, workspace=workspace)
        c.k, c.v = k, v
        assert torch.equal(got[:32], want[:32]) and torch.equal(got[40:], want[40:])
        assert torch.isfinite(got[:35]).all() and not torch.isfinite(got[35:40]).any()
    sv.sv_sync()
