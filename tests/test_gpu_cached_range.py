"""sv_attention_cached at the ends of its range: results at the end of F16's, keys by the hundred million."""
import math

import pytest
import torch

import cache_ref
from test_gpu_cached_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,have,prefix", [([1], 32, 0), ([1], 0, 32), ([40], 128, 0), ([20], 0, 128), ([200], 0, 128)])
@pytest.mark.parametrize("sign", [1, -1])
def test_values_at_the_end_of_f16(sv, n, have, prefix, sign):
    """A mean of equal values is that value, and finite: its error is one of 2^-11, which the largest F16 has no room for.

    Scores 0 and -ln 2 less a little: probabilities 2^8 and 128.07 (their head), of which F16 keeps 128.125, 4.3e-4
    more than the sum below; 65504 (1 + 2.4e-4) would round to infinity."""
    c = Case(n, [have], 1, 1, 64, prefix=prefix, e4m3=False, seed=1)
    tokens = have + prefix
    keys = torch.zeros(tokens, 1, 64, device="cuda", dtype=torch.float16)
    keys[1:, 0, 0] = -1.0
    places = c.b.places(0, -prefix, have)
    c.b.pool.store(0, *places, keys)
    c.b.pool.store(1, *places, torch.full_like(keys, sign * 65504.0))
    c.q.zero_()
    c.q[:, 0] = 1.0
    o = c.run(sv, scale=0.6926).double() * sign
    sv.sv_sync()
    # the formula's result is 65504; 2^-11 of it below, and no number above
    assert (o <= 65504).all() and (o >= 65504 * (1 - 2.0 ** -10)).all()


@pytest.mark.parametrize("own", [False, True])
def test_hundreds_of_millions_of_keys(sv, own):
    """A CTA works on its first item for more than the 2 s that a wait may last.

    One page, listed 2^20 times. Equal scores and values that are powers of two: every sum is exact (2^15 a tile of keys
    and 2^21 tiles at most), so that the mean is the value itself."""
    page, d, keys = 256, 8, 2 ** 28
    rows = 153 * (128 if own else 256)  # 153 items among 152 CTAs
    pool = torch.zeros(1, sv.sv_cache_page_bytes(page, 1, d), dtype=torch.uint8, device="cuda")
    k = torch.randn(page, d, generator=torch.Generator("cuda").manual_seed(1), device="cuda").half()
    v = torch.tensor([1.0, -0.5, 2.0, 0.25, -4.0, 8.0, 0.125, -1.0], device="cuda").half().expand(page, d).contiguous()
    pages = torch.zeros(keys // page, dtype=torch.int32, device="cuda")
    cache = sv.sv_cache(pool, 1, page, 1, d)
    full = torch.full((1,), page, dtype=torch.int32, device="cuda")
    sv.sv_cache_write(cache, sv.sv_cache_batch(1, pages, 1, full), k, v, None, page)
    lengths = torch.full((1,), keys if own else 0, dtype=torch.int32, device="cuda")
    batch = sv.sv_cache_batch(1, pages, keys // page if own else 0, lengths, None if own else pages, 0 if own else keys)
    q, o = (torch.zeros(rows, d, device="cuda", dtype=torch.float16) for _ in range(2))
    ws = torch.zeros(sv.sv_attention_cached_workspace(cache, batch, rows, 1), dtype=torch.uint8, device="cuda")
    sv.sv_attention_cached(cache, batch, q, o, None, rows, 1, workspace=ws)
    sv.sv_sync()
    assert torch.equal(o, v[:1].expand(rows, d))


@pytest.mark.parametrize("kind", ["prefix", "prefix of one tile", "own", "few", "few cut", "few over the prefix"])
@pytest.mark.parametrize("lg", [15, 17, 20])
@pytest.mark.parametrize("d,e4m3", [(64, False), (72, True), (128, True)])
def test_sums_over_many_keys(sv, kind, lg, d, e4m3):
    """Sums of the tensor cores, which truncate, are short: 2^lg keys of one CTA or warp (of several: cut) by way of one page,
    listed again and again.

    A product of 16 keys is added in two parts at most, each addition losing less than 2^-23 of the sum; over 16384 keys
    2^-12, beside the errors of bound()."""
    page, count, n = 256, 1, 1
    hk = {"prefix of one tile": 152, "few over the prefix": 1824}.get(kind, 1)
    if kind in ("few", "few cut"):
        count, n = (1824, 1) if kind == "few" else (100, 2)
    rows = {"prefix": 152 * 256, "prefix of one tile": 100, "own": 152 * 128, "few over the prefix": 1}.get(kind, count * n)
    c = Case([1], [page], hk, hk, d, page=page, e4m3=e4m3, seed=lg)
    g = torch.Generator("cuda").manual_seed(2)
    places = c.b.places(0, 0, page)
    c.b.pool.store(1, *places, (1 + torch.rand(page, hk, d, generator=g, device="cuda")).half())  # all of one sign
    n_keys = 2 ** lg
    pages = torch.full((count, n_keys // page), int(c.b.table[0, 0]), dtype=torch.int32, device="cuda")
    own = "prefix" not in kind
    lengths = torch.full((count,), n_keys if own else 0, dtype=torch.int32, device="cuda")
    batch = sv.sv_cache_batch(count, pages, n_keys // page if own else 0, lengths, None if own else pages, 0 if own else n_keys)
    cache = c.b.cache(sv)
    q = torch.randn(rows, hk * d, generator=g, device="cuda").half()
    o = torch.empty_like(q)
    ws = torch.zeros(sv.sv_attention_cached_workspace(cache, batch, rows, hk), dtype=torch.uint8, device="cuda")
    mask = 1 if kind == "few cut" else 0
    sv.sv_attention_cached(cache, batch, q, o, None, rows, hk, options=sv.sv_attention_options(mask=mask), workspace=ws)
    sv.sv_sync()
    k, v = c.b.sequence(0, 0), c.b.sequence(0, 1)
    some = torch.arange(0, rows, max(1, rows // 500), device="cuda")
    x = q[some].view(-1, hk, d)
    times = torch.full((len(some), 1, page), n_keys / page, dtype=torch.float64, device="cuda")  # a key's in the sequence
    if mask:  # the first query of two does not see the last key
        times[some % 2 == 0, :, -1] -= 1
    s = torch.einsum("rhd,khd->rhk", x.double(), k) / math.sqrt(d)
    terms = (torch.einsum("rhd,khd->rhk", x.double().abs(), k.abs()) / math.sqrt(d)).amax(-1, keepdim=True)
    p = times * torch.exp(s - s.amax(-1, keepdim=True))
    ref = torch.einsum("rhk,khd->rhd", p / p.sum(-1, keepdim=True), v)
    # (values of one sign: sum p |v| is the result)
    tol = cache_ref.bound(ref, ref, terms, page, float(v.abs().max()), d) + 2.0 ** -12 * ref
    assert ((o[some].double().view(ref.shape) - ref).abs() <= tol).all()
