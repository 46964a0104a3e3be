"""sv_attention_packed against the formulas in 64 bits (packed_ref: the tolerances' derivation stands at bound())."""
import math

import pytest
import torch

import packed_ref
from gpu_util import decode_e4m3

pytestmark = pytest.mark.gpu


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def _offsets(lens, start=0):
    return torch.tensor([start] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


class Case:
    """Inputs of one call: documents with lq queries and lk keys, optionally as columns of one projection's output,
    with rows before the first and behind the last document that belong to nobody."""

    def __init__(self, lq, lk, hq, hk, d, seed=0, fused=False, lead=0, tail=0, scale_q=1.0):
        self.lq, self.lk, self.hq, self.hk, self.d = lq, lk, hq, hk, d
        self.lead = lead
        self.tq, self.tk = lead + sum(lq) + tail, lead + sum(lk) + tail
        if fused:
            assert lq == lk
            width = (hq + 2 * hk) * d + 16
            qkv = _randn(seed, self.tq, width).half()
            self.q, self.k, self.v = (qkv[:, a * d:(a + h) * d] for a, h in ((0, hq), (hq, hk), (hq + hk, hk)))
        else:
            self.q = _randn(seed, self.tq, hq * d).half()
            self.k, self.v = _randn(seed + 1, self.tk, hk * d).half(), _randn(seed + 2, self.tk, hk * d).half()
        self.q.mul_(scale_q)
        self.q_off, self.k_off = _offsets(lq, lead), _offsets(lk, lead)

    def run(self, sv, out="f16", workspace=True, uniform=False, o=None, stream=None, **opt):
        prefix = opt.pop("prefix", None)
        if prefix is not None:
            prefix = torch.tensor(prefix, dtype=torch.int32).cuda()
        self.options = sv.sv_attention_options(prefix=prefix, **opt)
        if o is None:
            o = torch.full((self.tq, self.hq * self.d), 0x7F if out == "e4m3" else math.nan, device="cuda",
                           dtype=torch.uint8 if out == "e4m3" else torch.float16)
        ws = None
        if workspace is True:
            n = sv.sv_attention_packed_workspace(len(self.lq), self.tq, self.tk, self.hq, self.hk, self.d)
            ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        elif workspace is not False:
            ws = workspace
        self.ws = ws
        sv.sv_attention_packed(self.q, self.k, self.v, o, None if uniform else self.q_off,
                               None if uniform else self.k_off, len(self.lq), self.tq, self.tk, self.hq, self.hk,
                               self.d, q_stride=self.q.stride(0), k_stride=self.k.stride(0), v_stride=self.v.stride(0),
                               options=self.options, out_dtype=1 if out == "e4m3" else 0, workspace=ws, stream=stream)
        return o

    def docs(self):
        a = b = self.lead
        for n, (lq, lk) in enumerate(zip(self.lq, self.lk)):
            yield (n, a, lq, self.q[a:a + lq].reshape(lq, self.hq, self.d), self.k[b:b + lk].reshape(lk, self.hk, self.d),
                   self.v[b:b + lk].reshape(lk, self.hk, self.d))
            a, b = a + lq, b + lk

    def check(self, o, out="f16", mask=0, prefix=None, scale=None, softcap=0.0, slopes=None):
        got = decode_e4m3(o) if out == "e4m3" else o.double().cpu().numpy()
        got = torch.from_numpy(got)
        for n, a, lq, q, k, v in self.docs():
            if lq == 0:
                continue
            ref, av, terms = packed_ref.document(q, k, v, mask, prefix[n] if prefix is not None else 0, scale, softcap,
                                                 slopes)
            vmax = float(v.abs().max()) if v.numel() else 0.0
            tol = packed_ref.bound(ref, av, terms, k.shape[0], vmax, self.d, softcap, out == "e4m3")
            x = got[a:a + lq].reshape(ref.shape).cuda()
            assert torch.isfinite(x).all(), (n, "not finite")
            err = (x - ref).abs()
            assert (err <= tol).all(), (n, float((err - tol).max()), float(err.max()))
        # rows of no document
        rest = torch.cat([got[:self.lead], got[self.lead + sum(self.lq):]])
        assert torch.isnan(rest).all()


LENGTHS = [
    [1], [2, 1], [127], [128], [129], [64, 65, 63], [0, 5, 0, 0, 300, 1, 0], [255, 256, 257], [729, 730], [383, 1, 640],
    [17] * 40,
]


@pytest.mark.parametrize("lens", LENGTHS)
@pytest.mark.parametrize("hq,hk,d", [(3, 3, 72), (4, 2, 64), (2, 1, 128)])
def test_documents(sv, lens, hq, hk, d):
    c = Case(lens, lens, hq, hk, d, seed=sum(lens) + d, fused=True)
    c.check(c.run(sv))
    sv.sv_sync()


@pytest.mark.parametrize("lens", LENGTHS)
@pytest.mark.parametrize("hq,hk,d", [(3, 3, 72), (6, 2, 64), (4, 1, 128)])
def test_prefix_mask(sv, lens, hq, hk, d):
    c = Case(lens, lens, hq, hk, d, seed=sum(lens) + d)
    c.check(c.run(sv, mask=1), mask=1)
    prefix = [(7 * i + n) % (n + 3) for i, n in enumerate(lens)]
    c.check(c.run(sv, mask=1, prefix=prefix), mask=1, prefix=prefix)
    sv.sv_sync()


@pytest.mark.parametrize("d", [8, 16, 24, 40, 56, 64, 72, 80, 96, 104, 120, 128])
def test_head_widths(sv, d):
    c = Case([150, 33], [150, 290], 2, 2, d, seed=d)
    c.check(c.run(sv))
    c.check(c.run(sv, out="e4m3", mask=1), out="e4m3", mask=1)
    sv.sv_sync()


@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 2), (5, 1), (7, 1), (12, 4), (16, 1), (64, 1), (33, 1), (40, 8)])
def test_shared_key_heads(sv, hq, hk):
    c = Case([70, 1, 19], [70, 140, 300], hq, hk, 64, seed=hq)
    slopes = torch.linspace(0.0, 0.3, hq, device="cuda")
    c.check(c.run(sv, mask=1, slopes=slopes), mask=1, slopes=slopes)
    sv.sv_sync()


# unequal numbers of queries and keys: more keys (a cache), more queries (rows that see nothing), none of either
UNEQUAL = [([1], [1000]), ([1] * 7, [1, 64, 65, 129, 700, 2, 1023]), ([5, 3], [300, 4]), ([200], [50]),
           ([4, 9, 0], [0, 9, 30]), ([130, 20], [1, 513]), ([16] * 3, [2048, 100, 16]), ([1, 1], [0, 0]),
           ([1], [9000]), ([2, 1, 1], [4500, 33, 129])]


@pytest.mark.parametrize("lq,lk", UNEQUAL)
@pytest.mark.parametrize("mask", [0, 1])
@pytest.mark.parametrize("hq,hk,d", [(2, 2, 72), (8, 2, 128)])
def test_unequal_lengths(sv, lq, lk, mask, hq, hk, d):
    c = Case(lq, lk, hq, hk, d, seed=sum(lk))
    c.check(c.run(sv, mask=mask), mask=mask)
    c.check(c.run(sv, mask=mask, workspace=False), mask=mask)
    prefix = [3] * len(lq)
    c.check(c.run(sv, mask=1, prefix=prefix), mask=1, prefix=prefix)
    sv.sv_sync()


@pytest.mark.parametrize("cap,scale_q", [(30.0, 1.0), (30.0, 20.0), (5.0, 30.0), (0.25, 4.0), (500.0, 3.0)])
@pytest.mark.parametrize("lq,lk", [([300, 70], [300, 70]), ([1, 2], [700, 200])])
def test_softcap(sv, cap, scale_q, lq, lk):
    c = Case(lq, lk, 4, 2, 64, seed=int(cap), scale_q=scale_q)
    slopes = torch.tensor([0.5, 0.0, 0.01, 2.0], device="cuda")
    c.check(c.run(sv, softcap=cap), softcap=cap)
    c.check(c.run(sv, softcap=cap, mask=1, slopes=slopes), softcap=cap, mask=1, slopes=slopes)
    sv.sv_sync()


@pytest.mark.parametrize("lens", [[700], [130, 260, 9]])
def test_distance_bias(sv, lens):
    """Slopes of either sign, with and without the prefix mask."""
    c = Case(lens, lens, 4, 4, 72, seed=3, fused=True)
    slopes = torch.tensor([1.0, 0.125, 0.0, -0.05], device="cuda")
    c.check(c.run(sv, slopes=slopes), slopes=slopes)
    c.check(c.run(sv, slopes=slopes, mask=1, scale=0.3), slopes=slopes, mask=1, scale=0.3)
    sv.sv_sync()


@pytest.mark.parametrize("scale_q", [0.0, 40.0, 400.0])
def test_flat_and_steep_scores(sv, scale_q):
    """All scores equal, and scores in the hundreds (one key takes all)."""
    c = Case([200, 1], [200, 600], 2, 1, 64, seed=8, scale_q=scale_q)
    c.check(c.run(sv))
    sv.sv_sync()


def test_equal_documents_without_offsets(sv):
    c = Case([90] * 5, [90] * 5, 3, 3, 72, seed=2, fused=True)
    a, b = c.run(sv, uniform=True), c.run(sv)
    c.check(a)
    assert torch.equal(a, b)
    c = Case([1] * 6, [400] * 6, 4, 2, 64, seed=2)
    a, b = c.run(sv, uniform=True), c.run(sv)
    c.check(a)
    assert torch.equal(a, b)
    sv.sv_sync()


@pytest.mark.parametrize("out", ["f16", "e4m3"])
@pytest.mark.parametrize("lq,lk", [([140, 3], [140, 3]), ([1, 1], [300, 40])])
def test_rows_of_no_document_stay(sv, out, lq, lk):
    c = Case(lq, lk, 2, 2, 72, seed=4, lead=5, tail=9)
    c.check(c.run(sv, out=out), out=out)
    sv.sv_sync()


def test_large_values_saturate_in_e4m3(sv):
    c = Case([40], [40], 1, 1, 64, seed=4)
    c.v.mul_(100.0)
    o = c.run(sv, out="e4m3")
    sv.sv_sync()
    ref = packed_ref.document(*next(c.docs())[3:])[0].reshape(40, 64) * 16
    got = torch.from_numpy(decode_e4m3(o)).cuda() * 16
    assert (got[ref.abs() > 500].abs() == 448).all() and torch.isfinite(got).all()


def _by_rows(c, mask, prefix=0):
    """Row by row over the visible keys alone, so that hidden values cannot enter."""
    out = []
    for n, a, lq, q, k, v in c.docs():
        lim = packed_ref.limits(mask, lq, k.shape[0], prefix)
        for i in range(lq):
            out.append(packed_ref.document(q[i:i + 1], k[:lim[i]], v[:lim[i]])[0][0].reshape(-1) if lim[i]
                       else torch.zeros(c.hq * c.d, dtype=torch.float64, device="cuda"))
    return torch.stack(out)


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lq,lk,hidden", [
    ([60, 70], [60, 70], [45]),            # a later key of the first document
    ([150, 140], [150, 140], [149, 150]),  # the first document's last key, the second one's first
    ([3, 1], [200, 90], [198, 199]),       # few queries
    ([1, 1], [64, 300], [63, 64]),         # a neighbour's keys
])
def test_hidden_values_have_no_part(sv, poison, lq, lk, hidden):
    """NaN and infinities in keys and values reach the queries that see them, and no other."""
    mask = 1
    c = Case(lq, lk, 2, 1, 64, seed=21, lead=2, tail=3)
    clean = _by_rows(c, mask)
    rows = sum(lq)
    for what in (c.k, c.v):
        what[:2] = poison
        what[-3:] = poison
    for h in hidden:
        c.v[2 + h] = poison
        c.k[2 + h] = poison
    o = c.run(sv, mask=mask)
    sv.sv_sync()
    got = o[2:2 + rows].double()
    b = row = 0
    for a, n in zip(lq, lk):
        lim = packed_ref.limits(mask, a, n, 0)
        for i in range(a):
            sees = any(b <= h < b + lim[i] for h in hidden)
            if sees:
                # a score of NaN or +inf makes the row NaN; -inf times a query of either sign does as well
                assert not torch.isfinite(got[row]).all(), row
            else:
                assert torch.isfinite(got[row]).all(), row
                assert (got[row] - clean[row]).abs().max() <= 2.0 ** -9 * max(1.0, float(clean[row].abs().max())), row
            row += 1
        b += n


def test_same_bits_every_time_and_other_sizes_between(sv):
    """Repeated calls give the same bits, whatever ran on the workspace in between."""
    big = Case([1, 1, 1], [5000, 33, 9000], 8, 2, 128, seed=1)
    mid = Case([300, 200], [300, 200], 8, 2, 128, seed=2)
    n = sv.sv_attention_packed_workspace(3, big.tq, big.tk, 8, 2, 128)
    n = max(n, sv.sv_attention_packed_workspace(2, mid.tq, mid.tk, 8, 2, 128))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    a, b = big.run(sv, workspace=ws, mask=1), mid.run(sv, workspace=ws, mask=1)
    for _ in range(3):
        assert torch.equal(big.run(sv, workspace=ws, mask=1), a)
        assert torch.equal(mid.run(sv, workspace=ws, mask=1), b)
    sv.sv_sync()
    big.check(a, mask=1)
    mid.check(b, mask=1)


@pytest.mark.parametrize("lq,lk", [([200, 90], [200, 90]), ([1, 1, 1], [3000, 700, 40])])
def test_in_a_graph_and_on_two_streams(sv, lq, lk):
    """A captured call, replayed beside an eager one on another stream, each with a workspace of its own."""
    c = Case(lq, lk, 4, 2, 72, seed=6)
    want = c.run(sv, mask=1)
    o1, o2 = torch.zeros_like(want), torch.zeros_like(want)
    ws1, ws2 = torch.zeros_like(c.ws), torch.zeros_like(c.ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(sv, mask=1, o=o1, workspace=ws1)
    keep = c.options
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        g.replay()
        c.run(sv, mask=1, o=o2, workspace=ws2, stream=side)
    torch.cuda.synchronize()
    sv.sv_sync()
    assert torch.equal(o1, want) and torch.equal(o2, want)
    # offsets are read on the device: a replay follows them
    c.q_off.copy_(_offsets(lq[::-1]))
    c.k_off.copy_(_offsets(lk[::-1]))
    g.replay()
    eager = c.run(sv, mask=1)
    torch.cuda.synchronize()
    assert torch.equal(o1[:sum(lq)], eager[:sum(lq)])
    del keep


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("bad", [[0, 50, 40], [-7, 30, 40], [0, 30, 1000]])
def test_bad_offsets_are_reported(sv, which, bad):
    """Held inside the buffers on the device and reported by the next sv_sync; the context stays usable."""
    c = Case([30, 30], [30, 30], 2, 2, 64, seed=1)
    good = c.run(sv)
    sv.sv_sync()
    keep = getattr(c, which + "_off").clone()
    getattr(c, which + "_off").copy_(torch.tensor(bad, dtype=torch.int32))
    c.run(sv)
    with pytest.raises(sv.SvError) as e:
        sv.sv_sync()
    assert e.value.status == sv.SV_ERR_INVALID_ARG and "offsets" in str(e.value)
    getattr(c, which + "_off").copy_(keep)
    assert torch.equal(c.run(sv), good)
    sv.sv_sync()


def test_many_documents(sv):
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 40, (700,), generator=g).tolist()
    c = Case(lens, lens, 2, 2, 40, seed=7, fused=True)
    c.check(c.run(sv, mask=1), mask=1)
    keys = torch.randint(0, 200, (700,), generator=g).tolist()
    c = Case([1] * 700, keys, 2, 1, 64, seed=7)
    c.check(c.run(sv, mask=1), mask=1)
    sv.sv_sync()


def test_far_into_a_long_cache(sv):
    """Keys behind 2^31 values: row offsets pass 32 bits."""
    stride, n = 65536, 36000
    k = torch.empty(n * stride, dtype=torch.float16, device="cuda")[:n * stride].view(n, stride)
    d, lk = 64, [n - 700, 700]
    kv = _randn(3, n, 2 * d).half()
    k[:, 512:512 + 2 * d] = kv
    c = Case([1, 40], lk, 1, 1, d, seed=5)
    c.k, c.v = k[:, 512:512 + d], k[:, 512 + d:512 + 2 * d]
    c.tk = n
    c.check(c.run(sv, mask=1), mask=1)
    sv.sv_sync()


def test_projection_norm_rotation_attention_projection(sv):
    """The operators as they run together: fused projection, norm and rotation in place, packed attention, output
    projection with its residual, against the same chain in 64 bits rounded where the library stores F16."""
    lens, heads, d, width = [196, 729, 64], 16, 72, 1152
    rows = sum(lens)
    x = _randn(1, rows, width).half()
    w1, b1 = (_randn(2, 3 * width, width) / 34).half(), (_randn(3, 3 * width) * 0.1).half()
    w2, b2 = (_randn(4, width, width) / 34).half(), (_randn(5, width) * 0.1).half()
    gq, gk = (_randn(6, d) * 0.1 + 1).half(), (_randn(7, d) * 0.1 + 1).half()
    side = [14, 27, 8]
    pos = torch.cat([torch.stack([torch.arange(n * n) // n, torch.arange(n * n) % n]) for n in side], 1).int().cuda()
    plan = sv.sv_rope_plan_init(d, 2, sv.SV_ROPE_HALF, 100.0)
    qkv = torch.empty(rows, 3 * width, dtype=torch.float16, device="cuda")
    sv.sv_gemm_bias_act(x, w1, b1, None, 1, None, qkv, rows, 3 * width, width)
    raw = qkv.clone()
    q, k, v = qkv[:, :width], qkv[:, width:2 * width], qkv[:, 2 * width:]
    s = 3 * width
    sv.sv_qk_norm_rope(q, k, q, k, gq, gk, pos, plan, rows, heads, heads, d, q_stride=s, k_stride=s, q_out_stride=s,
                       k_out_stride=s)
    o = torch.empty(rows, width, dtype=torch.float16, device="cuda")
    off = _offsets(lens)
    ws = torch.zeros(sv.sv_attention_packed_workspace(3, rows, rows, heads, heads, d), dtype=torch.uint8, device="cuda")
    sv.sv_attention_packed(q, k, v, o, off, off, 3, rows, rows, heads, heads, d, q_stride=s, k_stride=s, v_stride=s,
                           workspace=ws)
    y = torch.empty(rows, width, dtype=torch.float16, device="cuda")
    sv.sv_gemm_bias_act(o, w2, b2, None, 1, x, y, rows, width, width)
    sv.sv_sync()

    import numpy as np
    import rope_ref
    ref = (x.double() @ w1.double().t() + b1.double())
    assert (raw.double() - ref).abs().max() <= 2.0 ** -10 * ref.abs().max()
    full = raw.double().cpu().numpy().reshape(rows, 3 * heads, d)
    parts = []
    for j, g in ((0, gq), (1, gk)):
        z = rope_ref.head_norm(full[:, j * heads:(j + 1) * heads], g.double().cpu().numpy(), 0, 1e-6)
        parts.append(torch.from_numpy(np.ascontiguousarray(rope_ref.rotate(z, pos.cpu().numpy(), d, 2, 0, 100.0)[0])))
    qr, kr = (p.half().cuda() for p in parts)
    vr = raw[:, 2 * width:].reshape(rows, heads, d)
    outs, a = [], 0
    for n in lens:
        outs.append(packed_ref.document(qr[a:a + n], kr[a:a + n], vr[a:a + n])[0].reshape(n, width))
        a += n
    oref = torch.cat(outs)
    # F16 operands one rounding apart move a score by up to 2^-11 of its terms (here below 1 in sum)
    assert (o.double() - oref).abs().max() <= 2.0 ** -8 * oref.abs().max()
    yref = oref @ w2.double().t() + b2.double() + x.double()
    assert (y.double() - yref).abs().max() <= 2.0 ** -8 * yref.abs().max()


# many rows over key ranges of more than 8 tiles of 128 keys, with few heads: the ranges are divided among the SMs
DIVIDED = [([40], [9000]), ([200, 3, 0], [5000, 40, 1500]), ([64, 64, 1], [3100, 0, 2300]), ([2500], [2500]),
           ([2300], [1500]), ([17] * 4, [1100, 1025, 2049, 4097])]


@pytest.mark.parametrize("lq,lk", DIVIDED)
@pytest.mark.parametrize("hq,hk,d,out", [(8, 2, 128, "f16"), (2, 1, 72, "e4m3"), (10, 1, 64, "f16")])
def test_divided_key_ranges(sv, lq, lk, hq, hk, d, out):
    c = Case(lq, lk, hq, hk, d, seed=sum(lk) + d, tail=3)
    c.check(c.run(sv, out=out), out=out)
    c.check(c.run(sv, out=out, mask=1), out=out, mask=1)
    prefix = [lk[0] // 2] * len(lq)
    slopes = torch.linspace(0.0, 0.01, hq, device="cuda")
    opt = dict(mask=1, prefix=prefix, slopes=slopes, softcap=4.0)
    c.check(c.run(sv, out=out, **opt), out=out, **opt)
    sv.sv_sync()


@pytest.mark.parametrize("poison", [math.nan, math.inf])
def test_hidden_values_in_divided_ranges(sv, poison):
    """A key hidden from some of the rows of a part, keys that no row sees, and a neighbour's keys."""
    lq, lk = [90, 60], [2600, 1300]
    c = Case(lq, lk, 2, 1, 64, seed=33, lead=2, tail=3)
    clean = _by_rows(c, 1)
    hidden = [2600 - 30, 2600 - 31, 2600 + 1299]
    for what in (c.k, c.v):
        what[:2] = poison
        what[-3:] = poison
        for h in hidden:
            what[2 + h] = poison
    got = c.run(sv, mask=1)[2:2 + sum(lq)].double()
    sv.sv_sync()
    sees = torch.tensor([i + 2600 - 90 >= 2600 - 31 for i in range(90)] + [i == 59 for i in range(60)], device="cuda")
    finite = torch.isfinite(got).all(1)
    assert torch.equal(finite, ~sees)
    err = (got - clean).abs()[~sees].amax(1)
    assert (err <= 2.0 ** -9 * clean[~sees].abs().amax(1).clamp(min=1.0)).all()


def test_divided_ranges_share_a_workspace(sv):
    """Calls of either kernel, divided and whole, one behind another on one workspace, eager and replayed: the same
    bits as with a workspace of their own."""
    cases = [Case([40], [9000], 8, 2, 128, seed=1), Case([1, 1], [7000, 300], 8, 2, 128, seed=2),
             Case([200, 3], [5000, 40], 2, 1, 72, seed=3), Case([300, 200], [300, 200], 4, 4, 64, seed=4),
             Case([1, 2], [6000, 9000], 4, 4, 72, seed=5)]
    want = [c.run(sv, mask=1) for c in cases]
    for c, o in zip(cases, want):
        c.check(o, mask=1)
    ws = torch.zeros(max(c.ws.numel() for c in cases), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(o) for o in want]
    for c, o in zip(cases, outs):
        c.run(sv, mask=1, workspace=ws, o=o)
    keep = []
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c, o in zip(cases[::-1], outs[::-1]):
            c.run(sv, mask=1, workspace=ws, o=o)
            keep.append(c.options)
    for _ in range(4):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    sv.sv_sync()


def test_runs_of_empty_documents(sv):
    """Documents without queries, without keys and without either, many in a row."""
    lq = [0] * 5 + [130] + [0] * 40 + [1] + [20, 30] + [0] * 33 + [260] + [0] * 3
    lk = [0, 9, 0, 0, 0] + [130] + [0, 3] * 20 + [5] + [0, 0] + [0] * 33 + [300] + [7] * 3
    for hq in (12, 3):  # many rows a document on average, few
        c = Case(lq, lk, hq, 3, 64, seed=6)
        for mask in (0, 1):
            c.check(c.run(sv, mask=mask), mask=mask)
            c.check(c.run(sv, mask=mask, workspace=False, out="e4m3"), mask=mask, out="e4m3")
    # items without keys one behind another, more than SMs
    c = Case([40] * 300, [0] * 299 + [200], 4, 4, 64, seed=6)
    c.check(c.run(sv, mask=1), mask=1)
    c = Case([1, 0, 0, 2] * 100, [0, 0, 70, 0] * 99 + [0, 0, 70, 9], 4, 4, 72, seed=6)
    c.check(c.run(sv), mask=0)
    # nothing but empty documents, and keys that nobody asks for
    c = Case([0] * 7 + [400], [0] * 8, 2, 2, 64, seed=6, tail=2)
    c.check(c.run(sv))
    c = Case([400, 3], [0, 0], 2, 2, 64, seed=6)
    c.check(c.run(sv, mask=1), mask=1)
    sv.sv_sync()


@pytest.mark.parametrize("group", [1, 3, 4, 5, 6, 12, 32, 33])
@pytest.mark.parametrize("d", [24, 64, 72, 128])
@pytest.mark.parametrize("out,pad", [("f16", 8), ("e4m3", 8), ("e4m3", 16)])
def test_output_rows(sv, group, d, out, pad):
    """Ways for a row to leave: whole warps of whole queries or not, on 16 bytes or not, with a row stride; the
    columns between the rows stay."""
    lq, lk = [70, 1, 150, 33], [70, 90, 150, 20]
    c = Case(lq, lk, 2 * group, 2, d, seed=group)
    width = 2 * group * d
    wide = torch.full((c.tq, width + pad), 0x7F if out == "e4m3" else math.nan, device="cuda",
                      dtype=torch.uint8 if out == "e4m3" else torch.float16)
    opt = sv.sv_attention_options(mask=1)
    sv.sv_attention_packed(c.q, c.k, c.v, wide, c.q_off, c.k_off, 4, c.tq, c.tk, 2 * group, 2, d, options=opt,
                           o_stride=width + pad, out_dtype=1 if out == "e4m3" else 0)
    sv.sv_sync()
    assert torch.equal(wide[:, width:].contiguous().view(torch.uint8),
                       torch.full_like(wide[:, width:].contiguous(), 0x7F if out == "e4m3" else math.nan).view(torch.uint8))
    c.check(wide[:, :width].contiguous(), out=out, mask=1)


@pytest.mark.parametrize("hk", [1, 2, 4, 6, 7])
@pytest.mark.parametrize("group,lq", [(1, [1, 1, 1, 1, 1]), (4, [3, 4, 1, 2, 4]), (1, [9, 1, 0, 30, 20])])
def test_few_rows_of_narrow_heads(sv, hk, group, lq):
    """Heads side by side in a block where there is much to read (the keys of documents cut anywhere), either number
    of row tiles, more rows in one document than a tile has."""
    lk = [9000, 17, 20000, 4001, 30003]
    c = Case(lq, lk, hk * group, hk, 72, seed=hk)
    a = c.run(sv, mask=1)
    c.check(a, mask=1)
    assert torch.equal(a, c.run(sv, mask=1, workspace=c.ws))
    slopes = torch.linspace(0.0, 0.002, hk * group, device="cuda")
    c.check(c.run(sv, out="e4m3", softcap=3.0, slopes=slopes), out="e4m3", softcap=3.0, slopes=slopes)
    c.check(c.run(sv, workspace=False))
    # a NaN that the first document's queries but its last do not see; all others of other documents do not either
    c.v[9000 - 1] = math.nan
    o = c.run(sv, mask=1)
    seen = lq[0] - 1
    assert not torch.isfinite(o[seen]).any()
    rest = torch.cat([o[:seen], o[seen + 1:]])
    assert torch.isfinite(rest).all()
    want = torch.cat([a[:seen], a[seen + 1:]])
    assert (rest.double() - want.double()).abs().max() <= 2.0 ** -9 * max(1.0, float(want.abs().max()))
    sv.sv_sync()


@pytest.mark.parametrize("hq,hk,d", [(8, 8, 128), (1, 1, 8), (16, 1, 64), (6, 6, 72)])
def test_one_row_over_a_very_long_range(sv, hq, hk, d):
    """One document's keys shared out among all blocks and joined."""
    c = Case([1], [70001], hq, hk, d, seed=9)
    a = c.run(sv)
    c.check(a)
    assert torch.equal(a, c.run(sv, workspace=c.ws))
    sv.sv_sync()


@pytest.mark.parametrize("hq,hk,d,out", [(2, 2, 64, "f16"), (4, 1, 72, "e4m3"), (2, 2, 72, "f16"), (3, 1, 128, "e4m3")])
@pytest.mark.parametrize("steps", [1, 40, 64, 200])
def test_rising_and_falling_scores(sv, hq, hk, d, out, steps):
    """Scores that rise by hundreds along the keys, evenly or in steps, so that a row's exponent is raised again and
    again, between tiles and inside them; and the same keys the other way round."""
    lens = [300, 70, 129]
    c = Case(lens, lens, hq, hk, d, seed=steps)
    u = torch.sign(_randn(steps + 1, d)).half()
    at = torch.cat([torch.arange(n) for n in lens]).cuda()
    ramp = (at // steps * steps).float()[:, None] / 25.0
    for flip in (False, True):
        c.q.copy_((u.float() + 0.05 * _randn(2, c.tq, hq, d)).reshape(c.tq, hq * d))
        c.k.copy_(((12.0 - ramp if flip else ramp)[:, None] * u.float() + 0.05 * _randn(3, c.tk, hk, d))
                  .reshape(c.tk, hk * d))
        c.check(c.run(sv, out=out), out=out)
        c.check(c.run(sv, out=out, mask=1), out=out, mask=1)
        slopes = torch.linspace(-0.1, 0.1, hq, device="cuda")
        c.check(c.run(sv, out=out, softcap=100.0, slopes=slopes), out=out, softcap=100.0, slopes=slopes)
    sv.sv_sync()


@pytest.mark.parametrize("d", [8, 24, 64, 72, 80, 104])
@pytest.mark.parametrize("out", ["f16", "e4m3"])
def test_bits_do_not_depend_on_the_call_before(sv, d, out):
    """What other calls leave on the SMs, NaN in every accumulator here, has no part in a result."""
    c = Case([300, 270, 513], [300, 270, 513], 48, 48, d, seed=d)
    clean = Case([300] * 4, [300] * 4, 48, 48, 128, seed=1)
    clean.run(sv)
    want = c.run(sv, out=out)
    c.check(want, out=out)
    clean.v.fill_(math.nan)
    assert torch.isnan(clean.run(sv)).all()
    assert torch.equal(c.run(sv, out=out).view(torch.uint8), want.view(torch.uint8))
    sv.sv_sync()


# Enough heads that items of two tiles fill the GPU (few heads: items of one tile, their keys shared out).
@pytest.mark.parametrize("heads,group,d", [(48, 1, 72), (80, 2, 64), (64, 4, 128), (90, 3, 40)])
@pytest.mark.parametrize("lens", [[300, 270, 513], [729], [129, 1, 0, 400], [640, 640]])
@pytest.mark.parametrize("out", ["f16", "e4m3"])
def test_many_heads(sv, heads, group, d, lens, out):
    c = Case(lens, lens, heads, heads // group, d, seed=heads, tail=2)
    c.check(c.run(sv, out=out), out=out)
    prefix = [n // 3 for n in lens]
    c.check(c.run(sv, out=out, mask=1, prefix=prefix), out=out, mask=1, prefix=prefix)
    slopes = torch.linspace(-0.01, 0.1, heads, device="cuda")
    for opt in (dict(slopes=slopes), dict(softcap=5.0, mask=1), dict(softcap=5.0, slopes=slopes, mask=1)):
        o = c.run(sv, out=out, **opt)
        c.check(o, out=out, **opt)
        assert torch.equal(o.view(torch.uint8), c.run(sv, out=out, workspace=c.ws, **opt).view(torch.uint8))
    sv.sv_sync()


@pytest.mark.parametrize("hq,hk,d", [(1, 1, 64), (4, 4, 72), (8, 2, 128), (5, 1, 24)])
@pytest.mark.parametrize("lq,lk", [([130], [1025]), ([1, 300], [1900, 300]), ([128], [1152]), ([700], [1024]),
                                   ([64, 0, 200], [2900, 130, 640]), ([150, 20], [2049, 4000]), ([140], [257])])
def test_few_items(sv, hq, hk, d, lq, lk):
    """Items of one tile whose key tiles are shared out between two groups: odd and even numbers of them, masks that
    leave one group's rows or both without keys, ranges that are divided among blocks as well."""
    c = Case(lq, lk, hq, hk, d, seed=d + sum(lk), lead=1, tail=4)
    slopes = torch.linspace(0.0, 0.05, hq, device="cuda")
    for opt in (dict(), dict(mask=1), dict(mask=1, prefix=[5] * len(lq), softcap=6.0), dict(slopes=slopes),
                dict(slopes=slopes, softcap=6.0, mask=1)):
        for out in ("f16", "e4m3"):
            o = c.run(sv, out=out, **opt)
            c.check(o, out=out, **opt)
            a = o.view(torch.uint8)
            assert torch.equal(a, c.run(sv, out=out, workspace=c.ws, **opt).view(torch.uint8))
    sv.sv_sync()


@pytest.mark.parametrize("poison", [math.nan, math.inf])
def test_hidden_values_among_few_items(sv, poison):
    """Keys that some rows see and others do not, in either group's tiles, and a neighbour's behind the last tile."""
    lq, lk = [200, 100], [1500, 900]
    c = Case(lq, lk, 1, 1, 64, seed=5, lead=2, tail=3)
    clean = _by_rows(c, 1)
    hidden = [[1350, 1470], [870]]
    for what in (c.k, c.v):
        what[:2] = poison
        what[-3:] = poison
        for h in hidden[0]:
            what[2 + h] = poison
        what[2 + 1500 + hidden[1][0]] = poison
    got = c.run(sv, mask=1)[2:2 + 300].double()
    sv.sv_sync()
    sees = torch.tensor([i + 1300 >= 1350 for i in range(200)] + [i + 800 >= 870 for i in range(100)], device="cuda")
    assert torch.equal(torch.isfinite(got).all(1), ~sees)
    err = (got - clean).abs()[~sees].amax(1)
    assert (err <= 2.0 ** -9 * clean[~sees].abs().amax(1).clamp(min=1.0)).all()


@pytest.mark.parametrize("rest", [100, 1100])
def test_long_ranges_among_many_documents(sv, rest):
    """Divided ranges in different groups of 32 documents, beside short ones."""
    lk = [rest] * 40
    lk[3], lk[35], lk[36], lk[20] = 9000, 7001, 0, 1025
    for hq, hk, d in ((1, 1, 72), (4, 2, 64)):
        c = Case([17] * 40, lk, hq, hk, d, seed=rest)
        for mask in (0, 1):
            o = c.run(sv, mask=mask)
            c.check(o, mask=mask)
            assert torch.equal(o, c.run(sv, mask=mask, workspace=c.ws))
    sv.sv_sync()


def test_more_parts_than_blocks(sv):
    """Items of one tile, divided into more parts than there are SMs."""
    for hq, hk, d in ((8, 2, 128), (6, 3, 64)):
        c = Case([1000], [9000], hq, hk, d, seed=d)
        for opt in (dict(), dict(mask=1), dict(mask=1, prefix=[4000], softcap=8.0)):
            o = c.run(sv, **opt)
            c.check(o, **opt)
            assert torch.equal(o, c.run(sv, workspace=c.ws, **opt))
    sv.sv_sync()


@pytest.mark.parametrize("few", [False, True])
def test_rows_far_behind_the_first(sv, few):
    """Queries, keys and output rows behind 2^31 values, for either kernel."""
    stride, n, d = 65536, 36000, 64
    wide = torch.empty(n * stride, dtype=torch.float16, device="cuda").view(n, stride)
    qkv = _randn(3, n, 3 * d).half()
    wide[:, 1024:1024 + 3 * d] = qkv
    lens = [1] * 17000 + [2] * 8000 + [3] * 1000 if few else [n - 500, 500]
    q_off = _offsets(lens)
    opt = sv.sv_attention_options(mask=1)
    sv.sv_attention_packed(wide[:, 1024:1024 + d], wide[:, 1024 + d:1024 + 2 * d], wide[:, 1024 + 2 * d:1024 + 3 * d],
                           wide[:, 2048:2048 + d], q_off, q_off, len(lens), n, n, 1, 1, d, q_stride=stride,
                           k_stride=stride, v_stride=stride, o_stride=stride, options=opt)
    sv.sv_sync()
    got = wide[:, 2048:2048 + d].double()
    a = 0
    for m in lens[:3] + lens[-40:] if few else lens:
        if few and a == 3:
            a = n - sum(lens[-40:])
        # (the last rows of a long document stand for all)
        rows = slice(max(0, m - 300), m)
        q, k, v = (qkv[a:a + m, i * d:(i + 1) * d].reshape(m, 1, d) for i in range(3))
        ref, av, terms = packed_ref.document(q[rows], k, v, 1)
        tol = packed_ref.bound(ref, av, terms, m, float(v.abs().max()), d)
        assert ((got[a:a + m][rows].reshape(ref.shape) - ref).abs() <= tol).all(), (a, m)
        a += m
