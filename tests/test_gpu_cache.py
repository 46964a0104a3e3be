"""sv_cache_write and sv_cache_read against the formulas: what is stored is compared byte for byte."""
import math

import pytest
import torch

import cache_ref

pytestmark = pytest.mark.gpu


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def _offsets(n, lead=0):
    return torch.tensor([lead] + n, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _expect(b, n, lead, k, v):
    """The pool after a write of the last n[i] tokens of every sequence from rows k, v [rows, heads, D]."""
    p = b.pool
    want = cache_ref.Pool(p.raw.shape[0], p.page, p.heads, p.dim, p.e4m3)
    want.raw.copy_(p.raw)
    row = lead
    for i, m in enumerate(n):
        if m:
            where = b.places(i, b.have[i] - m, b.have[i])
            for which, x in enumerate((k, v)):
                want.store(which, *where, x[row:row + m])
        row += m
    return want.raw


CASES = [  # own tokens, rows written of each, tokens of a page
    ([1], [1], 16), ([16], [16], 16), ([17, 15], [17, 15], 16), ([40, 7, 300], [1, 1, 1], 32), ([33, 0, 5, 0, 70], [2, 0, 5, 0, 33], 64),
    ([700], [513], 128), ([256, 257, 1], [255, 200, 1], 256), ([9] * 41, [3] * 41, 16), ([1000, 2000], [1000, 2000], 64),
]


@pytest.mark.parametrize("have,n,page", CASES)
@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 72), (8, 128)])
@pytest.mark.parametrize("e4m3", [True, False])
def test_write(sv, have, n, page, heads, dim, e4m3):
    """Everything else in the pages stays as it was."""
    b = cache_ref.Batch(have, page, heads, dim, e4m3=e4m3, seed=dim, fill=0x5A)
    lead, tail = 2, 3
    rows = lead + sum(n) + tail
    qkv = _randn(sum(have), rows, 3 * heads * dim + 8).half()  # columns of a fused projection
    qkv *= torch.exp(2.0 * _randn(1, rows, 1)).half()
    k, v = qkv[:, heads * dim:2 * heads * dim], qkv[:, 2 * heads * dim:3 * heads * dim]
    want = _expect(b, n, lead, k.reshape(rows, heads, dim), v.reshape(rows, heads, dim))
    sv.sv_cache_write(b.cache(sv), b.batch(sv), k, v, _offsets(n, lead), rows, k.stride(0), v.stride(0))
    sv.sv_sync()
    assert torch.equal(b.pool.raw, want)


@pytest.mark.parametrize("dim", [8, 16, 24, 40, 56, 64, 72, 80, 88, 96, 104, 112, 120, 128])
@pytest.mark.parametrize("e4m3", [True, False])
def test_head_widths_and_equal_rows(sv, dim, e4m3):
    """Without offsets every sequence has the same number of rows; and what was written comes back."""
    b = cache_ref.Batch([19, 5, 30], 16, 5, dim, e4m3=e4m3, seed=dim, fill=0)
    k, v = _randn(dim, 15, 5 * dim).half(), _randn(dim + 1, 15, 5 * dim).half()
    want = _expect(b, [5, 5, 5], 0, k.view(15, 5, dim), v.view(15, 5, dim))
    sv.sv_cache_write(b.cache(sv), b.batch(sv), k, v, None, 15)
    back = [torch.empty_like(k) for _ in range(2)]
    sv.sv_cache_read(b.cache(sv), b.batch(sv), *back, None, 15)
    sv.sv_sync()
    assert torch.equal(b.pool.raw, want)
    for x, y in zip((k, v), back):
        if not e4m3:
            assert torch.equal(x, y)
        else:  # 2^-4 of a value, or half a step of the subnormal codes: 2^-10 2^e, 448 2^e < 2 amax
            top = x.view(15, 5, dim).abs().amax(-1, keepdim=True).expand(15, 5, dim).reshape(15, -1).double()
            err = (x.double() - y.double()).abs()
            assert (err <= x.double().abs() * 2.0 ** -4 + top * 2.0 ** -9 / 224 * 0.5).all()


def test_special_values(sv):
    """Zeros, subnormal heads, the borders of the exponents and of the codes, F16's largest, infinities and NaN."""
    dim, heads = 64, 2
    rows = []
    for e in range(-15, 9):
        top = min(448.0 * 2.0 ** e, 65504.0)
        for x in (top, top * (1 + 2.0 ** -10), top * (1 - 2.0 ** -11), top * 0.501):
            row = torch.zeros(dim)
            row[:] = torch.linspace(-1, 1, dim) * x
            row[5], row[6] = x, -x / 3
            rows.append(row.clamp(-65504, 65504))
    ties = torch.cat([torch.arange(16, 32) / 16 + s for s in (0.03125, -0.03125)])  # halfway between codes
    rows.append(torch.cat([ties, -ties]))
    rows.append(torch.full((dim,), 2.0 ** -24))
    rows.append(torch.arange(dim) * 2.0 ** -24)
    rows.append(torch.zeros(dim))
    rows.append(-torch.zeros(dim))
    rows.append(torch.full((dim,), 65504.0))
    rows.append(torch.linspace(57344, 65504, dim))
    for x in (math.inf, -math.inf, math.nan):
        row = torch.ones(dim)
        row[dim - 1] = x
        rows.append(row)
    k = torch.stack(rows).half().cuda().repeat(1, heads)
    k[:, dim:] = k[:, dim:].flip(0)
    v = k.flip(0).contiguous()
    n = len(rows)
    for e4m3 in (True, False):
        b = cache_ref.Batch([n], 32, heads, dim, e4m3=e4m3)
        want = _expect(b, [n], 0, k.view(n, heads, dim), v.view(n, heads, dim))
        sv.sv_cache_write(b.cache(sv), b.batch(sv), k, v, None, n)
        back = [torch.empty_like(k) for _ in range(2)]
        sv.sv_cache_read(b.cache(sv), b.batch(sv), *back, None, n)
        sv.sv_sync()
        # (-0 is stored as such)
        assert torch.equal(b.pool.raw, want)
        for which in range(2):
            exact = b.sequence(0, which).view(n, -1)
            assert torch.equal(torch.isnan(exact), torch.isnan(back[which]))
            assert torch.equal(torch.nan_to_num(exact), torch.nan_to_num(back[which].double()))
            assert not torch.isinf(back[which]).any()


@pytest.mark.parametrize("have,n,prefix,page", [([5, 0, 40], [9, 4, 20], 21, 16), ([100], [829], 729, 64),
                                                ([3, 300], [0, 301], 1, 32), ([0], [256], 256, 256)])
@pytest.mark.parametrize("heads,dim", [(2, 72), (3, 128), (1, 40)])
@pytest.mark.parametrize("e4m3", [True, False])
def test_read_behind_a_prefix(sv, have, n, prefix, page, heads, dim, e4m3):
    """Exactly what is stored, into rows of any stride; other rows and columns stay."""
    b = cache_ref.Batch(have, page, heads, dim, prefix=prefix, e4m3=e4m3, seed=prefix)
    b.fill(dim)
    lead, tail = 1, 2
    rows = lead + sum(n) + tail
    out = torch.full((rows, 2 * heads * dim + 16), 7.0, device="cuda", dtype=torch.float16)
    k, v = out[:, 8:8 + heads * dim], out[:, 8 + heads * dim:8 + 2 * heads * dim]
    want = out.clone()
    row = lead
    for i, m in enumerate(n):
        for which in range(2):
            a = 8 + which * heads * dim
            want[row:row + m, a:a + heads * dim] = b.sequence(i, which)[len(b.sequence(i, which)) - m:].reshape(m, heads * dim).half()
        row += m
    sv.sv_cache_read(b.cache(sv), b.batch(sv), k, v, _offsets(n, lead), rows, k.stride(0), v.stride(0))
    sv.sv_sync()
    assert torch.equal(out, want)


def test_pages_behind_32_bits(sv):
    """A pool of 5 GB: pages whose places in it pass 2^32 bytes."""
    page, heads, dim = 256, 8, 128
    size = sv.sv_cache_page_bytes(page, heads, dim)
    first = (5 << 30) // size
    b = cache_ref.Batch([600, 30], page, heads, dim, prefix=10, seed=3, fill=0, first_page=first)
    n = [600, 30]
    k, v = _randn(1, 630, heads * dim).half(), _randn(2, 630, heads * dim).half()
    sv.sv_cache_write(b.cache(sv), b.batch(sv), k, v, _offsets(n), 630)
    back = [torch.empty_like(k) for _ in range(2)]
    sv.sv_cache_read(b.cache(sv), b.batch(sv), *back, _offsets(n), 630)
    sv.sv_sync()
    for which, x in enumerate((k, v)):
        codes, e, _ = cache_ref.quantise(x.view(630, heads, dim))
        exact = codes.double() * cache_ref.power(e).unsqueeze(-1)
        assert torch.equal(back[which].double(), exact.view(630, -1))
    assert int(b.pool.raw[:first].max()) == 0


@pytest.mark.parametrize("what", ["offsets", "beyond", "negative", "length", "short", "page", "low page"])
@pytest.mark.parametrize("read", [False, True])
def test_bad_sequences_are_reported(sv, what, read):
    """sv_sync reports them, the other sequences are served, and nothing is written out of place."""
    b = cache_ref.Batch([20, 30, 40], 16, 2, 64, seed=1, fill=0)
    b.fill(1)
    n = [4, 5, 6]
    off = _offsets(n)
    if what == "offsets":
        off[2] = 3
    elif what == "beyond":
        off[3] = 99
    elif what == "negative":
        off[0] = -1
    elif what == "length":
        b.lengths[1] = 16 * b.stride + 1
    elif what == "short":
        b.lengths[1] = 4
    elif what == "page":
        b.table[1, 1] = b.pool.raw.shape[0]
    else:
        b.table[1, 1] = -1
    before = b.pool.raw.clone()
    k, v = (torch.full((15, 128), 3.0, device="cuda", dtype=torch.float16) for _ in range(2))
    (sv.sv_cache_read if read else sv.sv_cache_write)(b.cache(sv), b.batch(sv), k, v, off, 15)
    with pytest.raises(sv.SvError) as e:
        sv.sv_sync()
    assert e.value.status == sv.SV_ERR_INVALID_ARG and "cache" in str(e.value)
    sv.sv_sync()
    if what in ("length", "short", "page", "low page"):
        if read:
            assert (k[4:9] == 3).all() and not (k[:4] == 3).all() and not (k[9:] == 3).all()
        else:
            want = b.pool.raw.clone()
            b.pool.raw.copy_(before)
            for i in (0, 2):
                for which in range(2):
                    b.pool.store(which, *b.places(i, b.have[i] - n[i], b.have[i]), k[:n[i]].view(-1, 2, 64))
            assert torch.equal(want, b.pool.raw)


def test_streams_and_graphs(sv):
    """Captured with the lengths in device memory: a replay writes at the place of the day."""
    b = cache_ref.Batch([40, 40], 16, 2, 64, seed=5, fill=0)
    cache, batch = b.cache(sv), b.batch(sv)
    k, v = _randn(1, 2, 128).half(), _randn(2, 2, 128).half()
    b.lengths.fill_(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.sv_cache_write(cache, batch, k, v, None, 2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sv_cache_write(cache, batch, k, v, None, 2)
        b.lengths.add_(1)
    for step in range(1, 40):
        k.copy_(_randn(100 + step, 2, 128).half())
        v.copy_(_randn(200 + step, 2, 128).half())
        graph.replay()
    back = [torch.empty(78, 128, device="cuda", dtype=torch.float16) for _ in range(2)]
    b.lengths.fill_(39)
    sv.sv_cache_read(cache, batch, *back, None, 78)
    sv.sv_sync()
    for which in range(2):
        for step in range(1, 40):
            x = _randn(100 * (which + 1) + step, 2, 128).half()
            codes, e, _ = cache_ref.quantise(x.view(2, 2, 64))
            exact = (codes.double() * cache_ref.power(e).unsqueeze(-1)).view(2, 128)
            for i in range(2):
                assert torch.equal(back[which][39 * i + step - 1].double(), exact[i])
