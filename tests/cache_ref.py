"""A paged key/value cache and attention over it in 64 bits, from the formulas (test helper)."""
import math

import torch

import packed_ref

MARK = 255


def power(e):
    """2^e in 64 bits, exactly (pow on the GPU may be off by its last bit)."""
    table = torch.tensor([2.0 ** k for k in range(-16, 240)], dtype=torch.float64, device=e.device)
    return table[(e + 16).long()]


def quantise(x):
    """x [..., D] in F16 -> (codes as E4M3, exponents e, marked heads): the least e in -15 .. 8 with max|x| <= 448 2^e."""
    y = x.double()
    bad = ~torch.isfinite(y).all(-1)
    y = torch.where(bad.unsqueeze(-1), torch.zeros_like(y), y)
    top = y.abs().amax(-1)
    e = torch.full(top.shape, -15, dtype=torch.int64, device=x.device)
    for k in range(-15, 8):
        e = torch.where(top > 448.0 * 2.0 ** k, torch.full_like(e, k + 1), e)
    z = y / power(e).unsqueeze(-1)
    z = torch.where(e.unsqueeze(-1) == 8, z.clamp(-240, 240), z)
    return z.float().to(torch.float8_e4m3fn), e, bad  # (F32 holds z: 11 bits and an exponent)


class Pool:
    """Pages as the library lays them out, with their parts as views."""

    def __init__(self, pages, page, heads, dim, e4m3=True, fill=0, device="cuda"):
        self.page, self.heads, self.dim, self.e4m3 = page, heads, dim, e4m3
        es = 1 if e4m3 else 2
        n, m = heads * page * dim * es, heads * page
        self.bytes = -(-2 * (n + m) // 128) * 128
        self.raw = torch.full((pages, self.bytes), fill, dtype=torch.uint8, device=device)
        self.codes = [self.raw[:, i * n:(i + 1) * n].unflatten(1, (heads, page, dim * es)) for i in range(2)]
        self.scales = [self.raw[:, 2 * n + i * m:2 * n + (i + 1) * m].unflatten(1, (heads, page)) for i in range(2)]

    def store(self, which, pages, at, x):
        """Heads x [tokens, heads, D] of keys (0) or values (1) at places `at` of `pages`."""
        if self.e4m3:
            codes, e, bad = quantise(x)
            codes, e = codes.view(torch.uint8), (e + 16).to(torch.uint8)
        else:
            bad = ~torch.isfinite(x).all(-1)
            codes = torch.where(bad.unsqueeze(-1), torch.zeros_like(x), x).contiguous().view(torch.uint8)
            e = torch.full(x.shape[:-1], 16, dtype=torch.uint8, device=x.device)
        self.codes[which][pages, :, at] = codes
        self.scales[which][pages, :, at] = torch.where(bad, torch.full_like(e, MARK), e)

    def values(self, which, pages, at):
        """What is stored there, in 64 bits [tokens, heads, D]."""
        codes = self.codes[which][pages, :, at].contiguous().view(torch.float8_e4m3fn if self.e4m3 else torch.float16)
        b = self.scales[which][pages, :, at].long().unsqueeze(-1)
        y = codes.double() * power(b - 16)
        return torch.where(b == MARK, torch.full_like(y, math.nan), y)


class Batch:
    """Sequences with `have` own tokens behind a prefix, their pages in no order, in a pool filled with `fill`."""

    def __init__(self, have, page, heads, dim, prefix=0, e4m3=True, seed=0, fill=0xFF, first_page=0, spare=2):
        g = torch.Generator("cuda").manual_seed(seed)
        self.have, self.prefix, self.page = have, prefix, page
        each = [-(-n // page) for n in have]
        pre = -(-prefix // page)
        self.pool = Pool(first_page + pre + sum(each) + spare, page, heads, dim, e4m3, fill)
        order = (torch.randperm(pre + sum(each) + spare, generator=g, device="cuda") + first_page).to(torch.int32)
        self.prefix_pages = order[:pre].contiguous() if pre else None
        self.stride = max(each + [1])
        self.table = torch.full((len(have), self.stride), -7, dtype=torch.int32, device="cuda")
        at = pre
        for i, n in enumerate(each):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.lengths = torch.tensor(have, dtype=torch.int32, device="cuda")

    def places(self, i, first, last):
        """(pages, places) of the tokens first .. last - 1 of sequence i, behind the prefix (which has negative ones)."""
        t = torch.arange(first, last, device="cuda")
        pages = torch.zeros_like(t)
        own = t >= 0
        pages[own] = self.table[i].long()[t[own] // self.page]
        if self.prefix:
            pages[~own] = self.prefix_pages.long()[(t[~own] + self.prefix) // self.page]
            t = torch.where(own, t, t + self.prefix)
        return pages, t % self.page

    def fill(self, seed=0, scale=1.0):
        """Random keys and values for every token of prefix and sequences."""
        g = torch.Generator("cuda").manual_seed(seed)
        p = self.pool
        spans = ([(0, -self.prefix, 0)] if self.prefix else []) + [(i, 0, n) for i, n in enumerate(self.have)]
        for i, a, b in spans:
            for which in range(2):
                x = torch.randn(b - a, p.heads, p.dim, generator=g, device="cuda")
                x *= torch.exp(torch.randn(b - a, p.heads, 1, generator=g, device="cuda"))  # heads of different sizes
                p.store(which, *self.places(i, a, b), (x * scale).clamp(-6e4, 6e4).half())

    def sequence(self, i, which):
        """Keys or values of prefix and own tokens, in 64 bits."""
        return self.pool.values(which, *self.places(i, -self.prefix, self.have[i]))

    def cache(self, sv):
        p = self.pool
        return sv.sv_cache(p.raw, p.raw.shape[0], p.page, p.heads, p.dim, sv.SV_DT_E4M3 if p.e4m3 else sv.SV_DT_F16)

    def batch(self, sv):
        return sv.sv_cache_batch(len(self.have), self.table, self.stride, self.lengths, self.prefix_pages, self.prefix)


def attention(q, k, v, own, causal, scale=None, softcap=0.0):
    """q [n, Hq, D] over k and v [prefix + own, Hk, D]: packed_ref's formula with the prefix visible to every query."""
    lk = k.shape[0]
    # (a document's queries stand at its last keys; a visible prefix of lk - own keys)
    return packed_ref.document(q, k, v, 1 if causal else 0, lk - own, scale, softcap)


def bound(o, a, terms, lk, vmax, d, softcap=0.0, e4m3=False):
    """packed_ref.bound; a value's factor in the exponent lets probabilities below 2^-14 lose 2^-33 * 448 * 2^e of the
    largest, and 448 * 2^e is below twice the head's largest magnitude, or 448 * 2^-15. The factor's addition rounds the
    exponent, |x| <= |score| + 15, once more (2^-24 of it, within the 8 operations and 2^-18 counted there)."""
    return packed_ref.bound(o, a, terms, lk, max(2 * vmax, 448 * 2.0 ** -15), d, softcap, e4m3)
