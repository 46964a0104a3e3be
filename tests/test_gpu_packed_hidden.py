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
