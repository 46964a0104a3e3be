"""The same call of sv_attention_cached, many times, gives the same bits: copies, operands and sums of tiles stay apart."""
import pytest
import torch

import cache_ref
from test_gpu_cached_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count,n,prefix,have,hq,hk,d,e4m3", [
    (256, 1, 32768, 100, 32, 8, 128, True),  # two tiles of rows over the prefix, CTAs that begin a second item
    (256, 1, 16384, 20, 16, 8, 64, True), (64, 2, 9000, 50, 12, 3, 96, True), (150, 1, 20000, 30, 8, 4, 128, False),
    (32, 1, 16384, 100, 32, 8, 128, True),   # one tile of rows
    (24, 5, 2047, 3000, 28, 4, 128, True), (8, 40, 0, 9000, 8, 4, 72, True), (6, 60, 300, 5000, 8, 4, 128, False)])
def test_same_bits(sv, count, n, prefix, have, hq, hk, d, e4m3):
    c = Case([n] * count, [have - (13 * i) % (have // 2 + 1) for i in range(count)], hq, hk, d, page=128, prefix=prefix, e4m3=e4m3,
             seed=count)
    ws = c.workspace(sv)
    want = c.run(sv, ws=ws, mask=1).clone()
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    o = torch.empty_like(want)
    for i in range(600):
        if i % 3 == 0:
            flush.fill_(i & 255)
        c.run(sv, ws=ws, o=o, mask=1)
        differ += (o != want).any()
    sv.sv_sync()
    assert int(differ) == 0
    # and the right ones: the first and last sequences against the formula
    rows = want.view(count, n, -1)
    for i in (0, count - 1):
        one = rows[i]
        ref, a, terms, lk, vmax = c.reference(i, i * n, True, None, 0.0)
        tol = cache_ref.bound(ref, a, terms, lk, vmax, d)
        assert ((one.double().view(ref.shape) - ref).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["pairs", "single", "own", "few"])
@pytest.mark.parametrize("d,e4m3", [(128, True), (72, True), (64, False)])
def test_same_bits_of_long_sequences(sv, kind, d, e4m3):
    """CTAs and warps that add up several runs or pieces of an item: pages listed many times over, in no order."""
    page, spare = 64, 500
    hk, rows, keys = {"pairs": (4, 600, 2 ** 20), "single": (8, 100, 2 ** 20), "own": (8, 256, 2 ** 20), "few": (2, 1, 2 ** 24 + 77)}[kind]
    c = Case([1], [page * spare], hk, hk, d, page=page, e4m3=e4m3, seed=5)
    g = torch.Generator("cuda").manual_seed(5)
    own = kind in ("own", "few")
    pages = c.b.table[0, torch.randint(0, spare, (-(-keys // page),), generator=g, device="cuda")].contiguous()
    lengths = torch.full((1,), keys if own else 0, dtype=torch.int32, device="cuda")
    cache = c.b.cache(sv)
    batch = sv.sv_cache_batch(1, pages, len(pages) if own else 0, lengths, None if own else pages, 0 if own else keys)
    q = torch.randn(rows, hk * d, generator=g, device="cuda").half()
    want, o = torch.empty_like(q), torch.empty_like(q)
    ws = torch.zeros(sv.sv_attention_cached_workspace(cache, batch, rows, hk), dtype=torch.uint8, device="cuda")
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    opt = sv.sv_attention_options(mask=1)
    sv.sv_attention_cached(cache, batch, q, want, None, rows, hk, options=opt, workspace=ws)
    for i in range(60):
        if i % 3 == 0:
            flush.fill_(i)
        sv.sv_attention_cached(cache, batch, q, o, None, rows, hk, options=opt, workspace=ws)
        differ += (o != want).any()
    sv.sv_sync()
    assert int(differ) == 0 and torch.isfinite(want).all()
