"""sv_attention_cached against the formulas in 64 bits (cache_ref: the tolerances' derivation stands at bound())."""
import math

import pytest
import torch

import cache_ref
from gpu_util import decode_e4m3

pytestmark = pytest.mark.gpu


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


class Case:
    """Queries n of each sequence over a prefix and their own `have` tokens; places that hold no token are 0xFF (NaN as
    E4M3 and as F16, a mark as a factor). Rows before the first and behind the last sequence belong to nobody."""

    def __init__(self, n, have, hq, hk, d, page=32, prefix=0, e4m3=True, seed=0, lead=0, tail=0, scale_q=1.0, wide=0,
                 first_page=0):
        self.n, self.hq, self.hk, self.d, self.lead = n, hq, hk, d, lead
        self.b = cache_ref.Batch(have, page, hk, d, prefix, e4m3, seed=seed, first_page=first_page)
        self.b.fill(seed)
        self.total = lead + sum(n) + tail
        q = _randn(seed + 7, self.total, hq * d + wide)
        self.q = (q * scale_q).half()[:, :hq * d]
        self.off = torch.tensor([lead] + n, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()

    def workspace(self, sv):
        size = sv.sv_attention_cached_workspace(self.b.cache(sv), self.b.batch(sv), self.total, self.hq)
        return torch.zeros(size, dtype=torch.uint8, device="cuda")

    def run(self, sv, out="f16", ws=None, o=None, uniform=False, stream=None, wide=0, **opt):
        if o is None:
            o = torch.full((self.total, self.hq * self.d + wide), 0x7F if out == "e4m3" else math.nan, device="cuda",
                           dtype=torch.uint8 if out == "e4m3" else torch.float16)
        self.kept = (self.b.cache(sv), self.b.batch(sv), sv.sv_attention_options(**opt), self.workspace(sv) if ws is None else ws)
        sv.sv_attention_cached(self.kept[0], self.kept[1], self.q, o, None if uniform else self.off, self.total, self.hq,
                               q_stride=self.q.stride(0), o_stride=o.stride(0), options=self.kept[2],
                               out_dtype=1 if out == "e4m3" else 0, workspace=self.kept[3], stream=stream)
        return o

    def reference(self, i, row, causal, scale, softcap):
        q = self.q[row:row + self.n[i]].reshape(-1, self.hq, self.d)
        k, v = self.b.sequence(i, 0), self.b.sequence(i, 1)
        ref, a, terms = cache_ref.attention(q, k, v, self.b.have[i], causal, scale, softcap)
        return ref, a, terms, len(k), float(v.abs().max()) if v.numel() else 0.0

    def check(self, o, out="f16", mask=0, scale=None, softcap=0.0):
        got = decode_e4m3(o) if out == "e4m3" else o.double().cpu().numpy()
        got = torch.from_numpy(got)
        row = self.lead
        for i, n in enumerate(self.n):
            if n:
                ref, a, terms, lk, vmax = self.reference(i, row, mask == 1, scale, softcap)
                tol = cache_ref.bound(ref, a, terms, lk, vmax, self.d, softcap, out == "e4m3")
                x = got[row:row + n, :self.hq * self.d].reshape(ref.shape).cuda()
                assert torch.isfinite(x).all(), (i, "not finite")
                if out == "e4m3":  # saturates at 28
                    ref = ref.clamp(-28, 28)
                err = (x - ref).abs()
                assert (err <= tol).all(), (i, float((err - tol).max()), float(err.max()))
            row += n
        rest = torch.cat([got[:self.lead], got[row:]])
        assert torch.isnan(rest).all()
        assert torch.isnan(got[:, self.hq * self.d:]).all()


LENGTHS = [  # queries, own tokens
    ([1], [1]), ([1], [0]), ([1, 1, 1], [15, 16, 17]), ([1, 1, 1, 1], [127, 128, 129, 0]), ([2, 1, 3], [64, 700, 65]),
    ([1] * 40, [(37 * i) % 300 for i in range(40)]), ([5, 0, 1, 9], [5, 40, 257, 1000]), ([3, 17], [1, 2]),
    ([1], [5000]), ([33, 70], [100, 512]),
]


@pytest.mark.parametrize("n,have", LENGTHS)
@pytest.mark.parametrize("hq,hk,d", [(3, 3, 72), (8, 2, 128), (7, 1, 64)])
@pytest.mark.parametrize("prefix", [0, 1, 129, 700])
@pytest.mark.parametrize("e4m3", [True, False])
def test_lengths(sv, n, have, hq, hk, d, prefix, e4m3):
    c = Case(n, have, hq, hk, d, page=16 if d == 72 else 64, prefix=prefix, e4m3=e4m3, seed=sum(have) + d, lead=1, tail=2)
    c.check(c.run(sv, mask=1), mask=1)
    sv.sv_sync()


@pytest.mark.parametrize("d", [8, 16, 24, 32, 40, 56, 64, 72, 80, 88, 96, 104, 120, 128])
@pytest.mark.parametrize("e4m3", [True, False])
def test_head_widths(sv, d, e4m3):
    c = Case([1, 2, 4], [150, 33, 290], 4, 2, d, prefix=45, e4m3=e4m3, seed=d, wide=8)
    c.check(c.run(sv, wide=16))
    c.check(c.run(sv, out="e4m3", mask=1), out="e4m3", mask=1)
    c = Case([70], [150], 4, 2, d, prefix=130, e4m3=e4m3, seed=d, wide=8)  # through tiles
    c.check(c.run(sv, wide=16, mask=1), mask=1)
    sv.sv_sync()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 2), (5, 1), (12, 4), (16, 1), (64, 1), (33, 1), (40, 8)])
@pytest.mark.parametrize("more", [1, 12])
@pytest.mark.parametrize("e4m3", [True, False])
def test_shared_heads_and_pages(sv, page, hq, hk, more, e4m3):
    c = Case([more, more, 3 * more], [70, 1, 400], hq, hk, 64, page=page, prefix=page + 3, e4m3=e4m3, seed=hq)
    c.check(c.run(sv, mask=1), mask=1)
    sv.sv_sync()


@pytest.mark.parametrize("prefix", [0, 300])
@pytest.mark.parametrize("scale,cap", [(0.0, 30.0), (0.3, 5.0), (0.02, 0.0), (0.0, 255.0), (0.0, 1000.0), (0.0, 1e30)])
def test_scale_and_cap(sv, prefix, scale, cap):
    c = Case([2, 1], [90, 333], 6, 3, 80, prefix=prefix, seed=4, scale_q=4.0)
    c.check(c.run(sv, scale=scale, softcap=cap), scale=scale or None, softcap=cap if cap < 1e29 else 0.0)
    sv.sv_sync()


@pytest.mark.parametrize("count,n,prefix,have", [(3, 1, 16411, 200), (40, 1, 2000, 37), (130, 2, 1000, 20), (1, 1, 20000, 0),
                                                 (70, 5, 513, 300)])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (4, 4, 72), (10, 2, 64)])
def test_batches_behind_a_long_prefix(sv, count, n, prefix, have, hq, hk, d):
    c = Case([n] * count, [(have * (i % 5)) // 4 for i in range(count)], hq, hk, d, page=64, prefix=prefix, seed=count)
    c.check(c.run(sv, mask=1, uniform=True), mask=1)
    c.check(c.run(sv, out="e4m3"), out="e4m3")
    sv.sv_sync()


@pytest.mark.parametrize("n,have", [([130, 1, 64], [130, 300, 1000]), ([9] * 50, [(61 * i) % 700 for i in range(50)]),
                                    ([40], [9000]), ([300], [20]), ([0, 50, 0, 0, 33], [5, 50, 700, 0, 2049])])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (4, 1, 72), (6, 2, 64), (5, 1, 96)])
@pytest.mark.parametrize("prefix,e4m3", [(0, True), (0, False), (300, True), (77, False)])
def test_many_rows(sv, n, have, hq, hk, d, prefix, e4m3):
    """Several queries of each sequence: rows in tiles of 128, those of a sequence among several, cut ranges."""
    c = Case(n, have, hq, hk, d, page=16 if hk == 1 else 64, prefix=prefix, e4m3=e4m3, seed=sum(have) + d, lead=1, tail=3, wide=8)
    c.check(c.run(sv, mask=1, wide=8), mask=1)
    c.check(c.run(sv, softcap=20.0, out="e4m3"), softcap=20.0, out="e4m3")
    sv.sv_sync()


@pytest.mark.parametrize("n", [[1, 2], [40, 0, 30]])
def test_no_own_pages(sv, n):
    """Sequences of the prefix alone: no page table at all."""
    c = Case(n, [0] * len(n), 4, 2, 72, prefix=150, seed=1)
    o, ws, cache, batch = torch.full((c.total, 288), math.nan, device="cuda", dtype=torch.float16), c.workspace(sv), c.b.cache(sv), c.b.batch(sv)
    batch.page_table, batch.table_stride = None, 0
    sv.sv_attention_cached(cache, batch, c.q, o, c.off, c.total, 4, options=sv.sv_attention_options(mask=1), workspace=ws)
    c.check(o, mask=1)
    sv.sv_sync()


def test_many_sequences(sv):
    """More than 32 times 32 sequences, empty ones among them, by either kernel."""
    for n, hq in ((1, 2), (40, 1)):
        count = 1100
        c = Case([n if i % 3 else 0 for i in range(count)], [(7 * i) % 50 for i in range(count)], hq, 1, 64, page=16, prefix=20, seed=n)
        c.check(c.run(sv, mask=1), mask=1)
    sv.sv_sync()


def test_uneven_long_caches(sv):
    """Ranges that are cut among CTAs, beside short ones and an empty one."""
    for hq, hk, d in ((8, 2, 128), (4, 4, 72), (16, 1, 64)):
        c = Case([1] * 6, [9000, 3, 0, 4097, 128, 20000], hq, hk, d, page=32, seed=d)
        c.check(c.run(sv))
        sv.sv_sync()


def test_large_scores(sv):
    """Rows whose maximum rises by far along the keys, and where one key outweighs all others."""
    c = Case([1, 4], [700, 300], 4, 2, 64, prefix=200, seed=9, scale_q=30.0)
    c.check(c.run(sv, mask=1), mask=1)
    sv.sv_sync()


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_marked_heads_among_many_rows(sv, e4m3, which, cap):
    """The same where a sequence's rows go through tiles: rows before a marked key have no part of it."""
    c = Case([60], [90], 4, 2, 64, prefix=200, e4m3=e4m3, seed=2)
    want = c.run(sv, mask=1, softcap=cap).view(60, 4, 64)
    spoiled = torch.ones(1, 2, 64, device="cuda", dtype=torch.float16)
    spoiled[0, 1, 7] = math.nan
    c.b.pool.store(which, *c.b.places(0, 53, 54), spoiled)  # queries 23 on see it, query heads 2 and 3 read its head
    got = c.run(sv, mask=1, softcap=cap).view(60, 4, 64)
    sv.sv_sync()
    bad = torch.zeros(60, 4, dtype=torch.bool, device="cuda")
    bad[23:, 2:] = True
    assert torch.equal(torch.isnan(got).all(-1), bad) and torch.equal(torch.isnan(got).any(-1), bad)
    assert torch.equal(got[:23], want[:23])


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("which", [0, 1])
def test_marked_heads(sv, e4m3, which):
    """A key or value that held a NaN makes the rows that see it NaN, in its head alone, and no others."""
    c = Case([3, 2], [50, 40], 4, 2, 64, prefix=20, e4m3=e4m3, seed=2)
    want = c.run(sv, mask=1)
    spoiled = torch.ones(1, 2, 64, device="cuda", dtype=torch.float16)
    spoiled[0, 1, 7] = math.nan
    # sequence 0: its last token but one; queries 1 and 2 see it, query heads 2 and 3 read its head
    c.b.pool.store(which, *c.b.places(0, 48, 49), spoiled)
    got = c.run(sv, mask=1).view(-1, 4, 64)
    sv.sv_sync()
    bad = torch.zeros(5, 4, dtype=torch.bool, device="cuda")
    bad[1:3, 2:] = True
    assert torch.equal(torch.isnan(got).all(-1), bad) and torch.equal(torch.isnan(got).any(-1), bad)
    # the others' bits, but for the spoiled head's value 1 where query 0 did not see the token before either
    same = ~bad
    same[1:3, :2] = False  # (they see the token's other head, which has changed)
    assert torch.equal(got[same], want.view(-1, 4, 64)[same])
    # in the prefix: every row of the head
    c = Case([3, 2], [50, 40], 4, 2, 64, prefix=20, e4m3=e4m3, seed=2)
    c.b.pool.store(which, *c.b.places(0, -1, 0), spoiled)
    got = c.run(sv, mask=1).view(-1, 4, 64)
    assert torch.isnan(got[:, 2:]).all() and not torch.isnan(got[:, :2]).any()


@pytest.mark.parametrize("n,have,hq", [([1] * 5, [90] * 5, 4), ([5], [90], 64), ([2, 1, 2], [700, 0, 1], 64)])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_query_of_nan(sv, n, have, hq, cap):
    """A query that holds an infinity or NaN spoils its own row alone."""
    c = Case(n, have, hq, 2, 64, prefix=140, seed=3)
    want = c.run(sv, softcap=cap).view(5, hq, 64)
    c.q[2, 64 + 5] = math.nan
    c.q[3, 3 * 64:4 * 64] = math.nan
    if not cap:
        c.q[3, 3 * 64:4 * 64] = math.inf  # (keys of both signs)
    got = c.run(sv, softcap=cap).view(5, hq, 64)
    bad = torch.zeros(5, hq, dtype=torch.bool, device="cuda")
    bad[2, 1] = bad[3, 3] = True
    assert torch.equal(torch.isnan(got).any(-1), bad)
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("n,hq", [([1], 2), ([40], 2)])
def test_query_of_infinity(sv, n, hq):
    """Scores of minus infinity alone leave 0 / 0, as the formula has it; with one of plus infinity the row is NaN too."""
    c = Case(n, [1], hq, 1, 64, e4m3=False, seed=3)
    key = torch.ones(1, 1, 64, device="cuda", dtype=torch.float16)
    key[0, 0, 1] = -1.0
    c.b.pool.store(0, *c.b.places(0, 0, 1), key)
    c.q[0, :64] = 0.0
    want = c.run(sv).view(-1, hq, 64)
    c.q[0, 0] = -math.inf
    c.q[0, 64 + 1] = -math.inf
    got = c.run(sv).view(-1, hq, 64)
    assert torch.isnan(got[0]).all() and torch.equal(got[1:], want[1:])
    sv.sv_sync()


def test_workspace_is_left_ready(sv):
    """One workspace for calls of several sizes in turn; the same call gives the same bits."""
    cases = [Case([1] * 7, [3000, 5, 0, 800, 90, 1, 4000], 8, 2, 128, prefix=900, seed=1),
             Case([40, 1], [300, 6000], 4, 4, 72, seed=2), Case([40, 1], [300, 6000], 8, 2, 128, prefix=77, seed=4),
             Case([300], [500], 4, 2, 64, seed=5), Case([2] * 30, [100] * 30, 8, 1, 64, prefix=5000, seed=3)]
    size = max(c.workspace(sv).numel() for c in cases)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    first = [c.run(sv, ws=ws, mask=1).clone() for c in cases]
    for _ in range(3):
        for c, want in zip(cases, first):
            assert torch.equal(c.run(sv, ws=ws, mask=1), want)
    for c in cases:
        c.check(c.run(sv, ws=ws, mask=1), mask=1)
    sv.sv_sync()


@pytest.mark.parametrize("what", ["offsets", "beyond", "length", "negative"])
@pytest.mark.parametrize("hq", [4, 80])
def test_bad_sequences_compute_nothing(sv, what, hq):
    c = Case([2, 1, 1], [40, 300, 20], hq, 2, 64, prefix=50, seed=1)
    if what == "offsets":
        c.off[1] = 4
    elif what == "beyond":
        c.off[3] = 77
    elif what == "length":
        c.b.lengths[1] = 32 * c.b.stride + 1
    else:
        c.b.lengths[0] = -1
    ws = c.workspace(sv)
    o = c.run(sv, ws=ws)
    with pytest.raises(sv.SvError) as e:
        sv.sv_sync()
    assert e.value.status == sv.SV_ERR_INVALID_ARG and "cache" in str(e.value)
    assert torch.isnan(o).all()
    c = Case([2, 1, 1], [40, 300, 20], hq, 2, 64, prefix=50, seed=1)
    c.check(c.run(sv, ws=ws))
    sv.sv_sync()


@pytest.mark.parametrize("where", ["own", "prefix"])
@pytest.mark.parametrize("page", [-1, 10 ** 9])
@pytest.mark.parametrize("hq", [4, 80])
def test_bad_pages_are_reported(sv, where, page, hq):
    """The other sequences' results stand."""
    c = Case([1, 1, 1], [100, 300, 20], hq, 2, 64, prefix=50, seed=1)
    want = c.run(sv)
    if where == "own":
        c.b.table[1, 3] = page
    else:
        c.b.prefix_pages[1] = page
    o = c.run(sv)
    with pytest.raises(sv.SvError) as e:
        sv.sv_sync()
    assert e.value.status == sv.SV_ERR_INVALID_ARG and "cache" in str(e.value)
    if where == "own":
        assert torch.equal(o[0], want[0]) and torch.equal(o[2], want[2])


@pytest.mark.parametrize("n", [[1] * 4, [30, 1, 9, 40]])
def test_streams_and_graphs(sv, n):
    """Two graphs with workspaces of their own replayed side by side, lengths that grow between replays."""
    cases = [Case(n, [200, 900, 30, 4000], 8, 2, 128, prefix=600, seed=i) for i in range(2)]
    streams, graphs, outs = [], [], []
    for c in cases:
        c.run(sv)
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        ws = c.workspace(sv)
        o = torch.empty(sum(n), 8 * 128, device="cuda", dtype=torch.float16)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            c.run(sv, ws=ws, o=o)
        streams.append(s), graphs.append(g), outs.append(o)
        c.keep = c.kept
    for have in ([200, 900, 30, 4000], [17, 0, 1, 3999], [200, 899, 30, 2500]):
        for c in cases:
            c.b.lengths.copy_(torch.tensor(have, dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(5):
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            c.b.have = have
            c.check(o)
    sv.sv_sync()


def test_pages_behind_32_bits(sv):
    size = sv.sv_cache_page_bytes(256, 8, 128)
    c = Case([1, 2], [600, 30], 16, 8, 128, page=256, prefix=300, seed=1, first_page=(5 << 30) // size)
    c.check(c.run(sv, mask=1), mask=1)
    sv.sv_sync()


def test_a_decoding_step(sv):
    """Norm and rotation, the cache's write, attention over it, as a decoder's layer runs them; then the same sequences
    read back and attended to as packed documents."""
    hq, hk, d, page, prefix = 8, 2, 128, 16, 90
    have = [33, 1, 160]
    b = cache_ref.Batch(have, page, hk, d, prefix, seed=1)
    b.fill(1, scale=0.5)
    qkv = _randn(5, 3, (hq + 2 * hk) * d).half()
    q, k, v = qkv[:, :hq * d], qkv[:, hq * d:(hq + hk) * d], qkv[:, (hq + hk) * d:]
    gamma = torch.ones(d, device="cuda", dtype=torch.float16)
    plan = sv.sv_rope_plan_init(d)
    pos = (b.lengths + prefix - 1).view(1, 3)
    sv.sv_qk_norm_rope(q, k, q, k, gamma, gamma, pos, plan, 3, hq, hk, d, q_stride=q.stride(0), k_stride=k.stride(0),
                       q_out_stride=q.stride(0), k_out_stride=k.stride(0))
    cache, batch = b.cache(sv), b.batch(sv)
    sv.sv_cache_write(cache, batch, k, v, None, 3, k.stride(0), v.stride(0))
    o = torch.empty(3, hq * d, device="cuda", dtype=torch.float16)
    ws = torch.zeros(sv.sv_attention_cached_workspace(cache, batch, 3, hq), dtype=torch.uint8, device="cuda")
    opt = sv.sv_attention_options(mask=1)
    sv.sv_attention_cached(cache, batch, q, o, None, 3, hq, q_stride=q.stride(0), options=opt, workspace=ws)
    lens = [prefix + n for n in have]
    k_off = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    kk, vv = (torch.empty(sum(lens), hk * d, device="cuda", dtype=torch.float16) for _ in range(2))
    sv.sv_cache_read(cache, batch, kk, vv, k_off, sum(lens))
    packed = torch.empty_like(o)
    sv.sv_attention_packed(q, kk, vv, packed, None, k_off, 3, 3, sum(lens), hq, hk, d, q_stride=q.stride(0), options=opt)
    sv.sv_sync()
    row = 0
    for i, n in enumerate(lens):
        kd, vd = b.sequence(i, 0), b.sequence(i, 1)
        assert torch.equal(kk[row:row + n].double(), kd.reshape(n, -1)) and torch.equal(vv[row:row + n].double(), vd.reshape(n, -1))
        ref, a, terms = cache_ref.attention(q[i:i + 1].reshape(1, hq, d), kd, vd, have[i], True)
        tol = cache_ref.bound(ref, a, terms, n, float(vd.abs().max()), d)
        for x in (o, packed):
            assert ((x[i].double().view(1, hq, d) - ref).abs() <= tol).all()
        row += n
