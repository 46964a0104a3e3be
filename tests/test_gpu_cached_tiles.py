"""sv_attention_cached where rows go through tiles: infinite scores under a cap, marked heads in the prefix, scales and
caps, pages behind 32 bits."""
import math

import pytest
import torch

import cache_ref
from test_gpu_cached_attention import Case

pytestmark = pytest.mark.gpu

# queries, own tokens of each sequence: few rows; one tile of rows over the prefix; two, and tiles over the own tokens
FEW, ONE, TWO = ([1, 2], [50, 40]), ([20, 10], [50, 40]), ([90, 80], [150, 40])


@pytest.mark.parametrize("n,have", [FEW, ONE, TWO])
@pytest.mark.parametrize("prefix", [140, 141, 142, 143, 257, 515])
@pytest.mark.parametrize("e4m3", [True, False])
def test_infinite_scores_under_a_cap(sv, n, have, prefix, e4m3):
    """Scores of an infinity are the cap or its negative, wherever the prefix ends; other rows keep their bits."""
    cap, at = 20.0, 5
    c = Case(n, have, 6, 3, 64, prefix=prefix, e4m3=e4m3, seed=prefix)
    g = torch.Generator("cuda").manual_seed(1)
    for i, a, b in [(0, -prefix, 0)] + [(i, 0, h) for i, h in enumerate(have)]:
        keys = torch.randn(b - a, 3, 64, generator=g, device="cuda")
        keys[..., at] = torch.where(torch.rand(b - a, 3, generator=g, device="cuda") < 0.5, -1.0, 1.0)  # never 0
        c.b.pool.store(0, *c.b.places(i, a, b), keys.half())
    want = c.run(sv, mask=1, softcap=cap).view(-1, 6, 64)
    q = c.q.view(-1, 6, 64)
    rows = [(0, 1, math.inf), (sum(n) - 1, 4, -math.inf)]
    for row, head, x in rows:
        q[row, head, at] = x
    got = c.run(sv, mask=1, softcap=cap).view(-1, 6, 64)
    sv.sv_sync()
    same = torch.ones(sum(n), 6, dtype=torch.bool, device="cuda")
    for row, head, _ in rows:
        same[row, head] = False
    assert torch.equal(got[same], want[same])
    first = 0
    for i, m in enumerate(n):
        ref, a, terms, lk, vmax = c.reference(i, first, True, None, cap)
        # a capped infinity is exact but for the cap's own error
        tol = cache_ref.bound(ref, a, torch.where(torch.isinf(terms), 0.0, terms), lk, vmax, 64, cap)
        err = (got[first:first + m].double() - ref).abs()
        assert torch.isfinite(got[first:first + m]).all() and (err <= tol).all(), float((err - tol).max())
        first += m


@pytest.mark.parametrize("n,have", [ONE, TWO])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("at", [-1, -130, -300])
def test_marked_heads_in_the_prefix(sv, n, have, which, cap, e4m3, at):
    """Every row of the head that reads it is NaN, the others keep their bits."""
    c = Case(n, have, 4, 2, 64, prefix=300, e4m3=e4m3, seed=2)
    x = torch.ones(1, 2, 64, device="cuda", dtype=torch.float16)
    c.b.pool.store(which, *c.b.places(0, at, at + 1), x)
    want = c.run(sv, mask=1, softcap=cap).view(-1, 4, 64)
    assert torch.isfinite(want).all()
    x[0, 1, 7] = math.inf
    c.b.pool.store(which, *c.b.places(0, at, at + 1), x)
    got = c.run(sv, mask=1, softcap=cap).view(-1, 4, 64)
    sv.sv_sync()
    assert torch.isnan(got[:, 2:]).all() and torch.equal(got[:, :2], want[:, :2])


@pytest.mark.parametrize("n,have,prefix", [(*ONE, 300), (*TWO, 300), ([60], [333], 0)])
@pytest.mark.parametrize("scale,cap", [(0.0, 30.0), (0.3, 5.0), (0.02, 0.0), (0.0, 255.0), (0.0, 1000.0), (0.05, 300.0), (0.0, 1e30)])
@pytest.mark.parametrize("e4m3", [True, False])
def test_scale_and_cap(sv, n, have, prefix, scale, cap, e4m3):
    c = Case(n, have, 6, 3, 80, prefix=prefix, e4m3=e4m3, seed=4, scale_q=4.0)
    c.check(c.run(sv, scale=scale, softcap=cap, mask=1), mask=1, scale=scale or None, softcap=cap if cap < 1e29 else 0.0)
    sv.sv_sync()


@pytest.mark.parametrize("n", [[20, 10], [70, 60]])
@pytest.mark.parametrize("e4m3", [True, False])
def test_pages_behind_32_bits(sv, n, e4m3):
    """A pool of more than 5 GB, by bulk copies and by the tensor map."""
    size = sv.sv_cache_page_bytes(256, 8, 128, 1 if e4m3 else 0)
    c = Case(n, [600, 30], 16, 8, 128, page=256, prefix=300, e4m3=e4m3, seed=1, first_page=(5 << 30) // size)
    c.check(c.run(sv, mask=1), mask=1)
    sv.sv_sync()


@pytest.mark.parametrize("n,have", [FEW, ONE, TWO])
def test_workspace_behind_its_counters(sv, n, have):
    """Only the first 4096 bytes have to be zero before the first use."""
    c = Case(n, have, 8, 2, 128, prefix=700, seed=3)
    ws = c.workspace(sv)
    want = c.run(sv, ws=ws, mask=1)
    other = torch.full_like(ws, 0xFF)
    other[:4096] = 0
    assert torch.equal(c.run(sv, ws=other, mask=1), want)
    assert torch.equal(c.run(sv, ws=other, mask=1), want)
    sv.sv_sync()
