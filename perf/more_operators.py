"""Cases for measuring the operators on a paged key/value cache: writing it, reading it back, and attention over it for
a batch whose sequences may share a prefix.

``run`` computes a case in plain torch operations, or, with ``own`` set, through the library's
entry points: ``sv_cache_write``, ``sv_cache_read`` and ``sv_attention_cached``.

A page holds ``page`` tokens: the keys of every head [heads, page, head_dim], the values likewise, and a byte for each
token and head of the keys and of the values, b: what is stored counts 2^(b - 16). E4M3 caches take the least scale
2^-15 .. 2^8 with which the largest magnitude of the head is at most 448, F16 caches 2^0.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------- cases

def _move(name, op, seqs, n_min, n_max, own_min, own_max, mix, prefix, kv_heads, head_dim, page, dtype):
    """Each sequence's last n_min..n_max tokens (n_max 0: all) of own_min..own_max, written or read; prefix: read too."""
    return {"name": name, "op": op, "seqs": seqs, "n_min": n_min, "n_max": n_max, "own_min": own_min, "own_max": own_max,
            "mix": mix, "prefix": prefix, "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "dtype": dtype}


def _attn(name, seqs, n_min, n_max, own_min, own_max, mix, prefix, heads, kv_heads, head_dim, page, dtype,
          mask="prefix", softcap=0.0, out="f16"):
    """n_min..n_max queries of each sequence over the shared prefix and its own_min..own_max tokens."""
    return {"name": name, "op": "attention", "seqs": seqs, "n_min": n_min, "n_max": n_max, "own_min": own_min,
            "own_max": own_max, "mix": mix, "prefix": prefix, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "dtype": dtype, "mask": mask, "softcap": softcap, "out": out}


def listed():
    return [
        # the new token of each of 64 requests in a decoding step: a call's latency
        _move("write_step", "write", 64, 1, 1, 30, 2000, 1, 0, 8, 128, 64, "e4m3"),
        # six prompts, from the columns of a fused projection
        _move("write_prompts", "write", 6, 0, 0, 900, 5003, 2, 0, 8, 128, 64, "e4m3"),
        # the tokens of 32 images of 378 px as keys of 16 heads of 72, unquantised, small pages
        _move("write_images", "write", 32, 0, 0, 729, 729, 3, 0, 16, 72, 16, "f16"),
        # one image's tokens back, for a pass over the packed rows
        _move("read_image", "read", 1, 0, 0, 729, 729, 4, 0, 16, 72, 32, "e4m3"),
        # conversations whole, the shared image prefix among them, to go on in a long prompt pass
        _move("read_prompts", "read", 5, 0, 0, 500, 9001, 5, 729, 8, 128, 64, "e4m3"),
        # four short requests, nothing shared: a call's latency
        _attn("attn_short", 4, 1, 1, 60, 700, 6, 0, 16, 16, 72, 32, "e4m3"),
        # one new token of 16 requests over long caches of their own
        _attn("attn_long", 16, 1, 1, 900, 32768, 9, 0, 32, 8, 128, 64, "e4m3"),
        # three continuations of one long document
        _attn("attn_document", 3, 1, 1, 20, 300, 7, 16411, 32, 8, 128, 64, "e4m3"),
        # 32 requests behind the same instructions
        _attn("attn_shared", 32, 1, 1, 30, 1000, 8, 8192, 32, 8, 128, 64, "e4m3"),
        # five drafted tokens of each of 24 requests checked at once, output for an E4M3 projection
        _attn("attn_draft", 24, 5, 5, 200, 3000, 10, 2047, 28, 4, 128, 128, "e4m3", out="e4m3"),
        # 64 requests, unquantised cache, capped scores, narrow heads of their own
        _attn("attn_capped", 64, 1, 1, 40, 900, 11, 4096, 12, 12, 64, 16, "f16", softcap=30.0),
        # 256 samples of one long prompt
        _attn("attn_samples", 256, 1, 1, 16, 512, 12, 32768, 32, 8, 128, 128, "e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention", "attention"])
    head_dim = rng.choice([64, 72, 80, 96, 128])
    page, dtype = rng.choice([16, 32, 64, 128]), rng.choice(["e4m3", "e4m3", "f16"])
    mix = rng.randint(0, 9999)
    if op != "attention":
        own_max = _log(rng, 1, 9000)
        seqs = _log(rng, 1, max(1, min(256, 24000 // own_max)))
        n = rng.choice([0, 0, 1, min(own_max, 7)])
        own_min = max(1, n, own_max // 6)
        prefix = rng.choice([0, 100, 729]) if op == "read" else 0
        c = _move("", op, seqs, n, n, own_min, own_max, mix, prefix, rng.randint(1, 16), head_dim, page, dtype)
    else:
        group = rng.choice([1, 1, 2, 4, 4, 5, 7, 8])
        kv = rng.randint(1, 32 // group if group > 1 else 16)
        prefix = rng.choice([0, _log(rng, 40, 32768), _log(rng, 40, 32768)])
        n = rng.choice([1, 1, 1, 2, 5, 8])
        own_max = max(n, _log(rng, 1, 16000))
        most = min(256, (1 << 28) // (own_max * kv * head_dim * (1 if dtype == "e4m3" else 2)),
                   (1 << 30) // ((prefix + own_max) * n * kv * group * head_dim // 32 + 1))
        seqs = _log(rng, 1, max(1, most))
        c = _attn("", seqs, n, n, max(n, own_max // 6), own_max, mix, prefix, kv * group, kv, head_dim, page, dtype,
                  rng.choice(["document", "prefix", "prefix"]), rng.choice([0.0, 0.0, 0.0, 30.0, 50.0]),
                  rng.choice(["f16", "f16", "f16", "e4m3"]))
    del c["name"]
    return c


def _lengths(c):
    """(tokens of the call, own tokens of the cache) of every sequence."""
    r = random.Random(c["mix"])
    have = [r.randint(c["own_min"], c["own_max"]) for _ in range(c["seqs"])]
    if c["n_max"]:
        return [r.randint(c["n_min"], c["n_max"]) for _ in have], have
    return [h + (c["prefix"] if c["op"] == "read" else 0) for h in have], have


def _pages(c):
    """(pages of the prefix, pages of the longest sequence's own tokens, pages of the cache)."""
    _, have = _lengths(c)
    prefix = -(-c["prefix"] // c["page"])
    each = [-(-h // c["page"]) for h in have]
    return prefix, max(each), prefix + sum(each) + 3


def work(c):
    n, have = _lengths(c)
    es = 1 if c["dtype"] == "e4m3" else 2
    head = c["kv_heads"] * 2  # keys and values
    stored = c["head_dim"] * es + 1
    if c["op"] != "attention":
        return {"bytes": sum(n) * head * (stored + 2 * c["head_dim"]), "flops": 2 * sum(n) * head * c["head_dim"]}
    seen = 0
    for a, b in zip(n, have):
        seen += a * (c["prefix"] + b)
        if c["mask"] == "prefix":
            seen -= sum(min(b, x) for x in range(a))
    rows = sum(n) * c["heads"] * c["head_dim"]
    return {"bytes": (c["prefix"] + sum(have)) * head * stored + rows * (3 if c["out"] == "e4m3" else 4),
            "flops": 4 * seen * c["heads"] * c["head_dim"]}


# ---------------------------------------------------------------- inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _shift(amax):
    """The least exponent -15 .. 8 with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax == 0, torch.full_like(e, -15), e.clamp_min(-15))


def _quantise(x, dtype):
    """x in 32 bits [..., head_dim] as it is stored (raw bytes, last dimension in bytes) and its scale's bytes."""
    if dtype == "f16":
        return x.half().view(torch.uint8), torch.full(x.shape[:-1], 16, device=x.device, dtype=torch.uint8)
    e = _shift(x.abs().amax(-1))
    most = torch.where(e == 8, 240.0, 448.0).unsqueeze(-1)  # 256 * 2^8 is beyond F16
    y = torch.ldexp(x, -e.unsqueeze(-1))
    y = torch.minimum(torch.maximum(y, -most), most).to(torch.float8_e4m3fn)
    return y.view(torch.uint8), (e + 16).to(torch.uint8)


def _layout(c):
    """Bytes of a page: of its keys (and of its values), of their scales, of the whole."""
    codes = c["kv_heads"] * c["page"] * c["head_dim"] * (1 if c["dtype"] == "e4m3" else 2)
    scales = c["kv_heads"] * c["page"]
    return codes, scales, -(-2 * (codes + scales) // 128) * 128


def _parts(c, pool):
    """The stored bytes of keys and values [pages, heads, page, bytes of a head], and their scales [pages, heads, page]."""
    codes, scales, _ = _layout(c)
    h, p = c["kv_heads"], c["page"]

    def part(at, n, *shape):
        return pool[:, at:at + n].unflatten(1, shape)

    return (part(0, codes, h, p, codes // scales), part(codes, codes, h, p, codes // scales),
            part(2 * codes, scales, h, p), part(2 * codes + scales, scales, h, p))


def _inputs(c, seed):
    """The inputs of a case, made from the seed."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, have = _lengths(c)
    h, d, page = c["kv_heads"], c["head_dim"], c["page"]
    prefix_pages, table_pages, pages = _pages(c)
    s = {}
    # pages of a pool that has been in use for some time: in no order
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    s["prefix_pages"] = order[:prefix_pages].contiguous() if prefix_pages else None
    s["table"] = torch.full((c["seqs"], table_pages), -1, device=DEV, dtype=torch.int32)
    at = prefix_pages
    for i, x in enumerate(have):
        k = -(-x // page)
        s["table"][i, :k] = order[at:at + k]
        at += k
    s["lengths"] = torch.tensor(have, device=DEV, dtype=torch.int32)
    s["offsets"] = torch.tensor([0] + n, device=DEV).cumsum(0).to(torch.int32)
    s["pool"] = torch.zeros(pages, _layout(c)[2], device=DEV, dtype=torch.uint8)
    # a few dimensions of the keys much larger than the others, heads of different sizes
    spread = torch.exp(0.5 * _normal(g, h, 1)) * (1.0 + 4.0 * (torch.rand(h, d, generator=g, device=DEV) < 0.04))
    if c["op"] == "write":
        qkv = _normal(g, sum(n), 4 * h * d).half()  # queries of twice as many heads beside them
        s["k"], s["v"] = qkv[:, 2 * h * d:3 * h * d], qkv[:, 3 * h * d:]
        s["k"].mul_(spread.half().view(-1))
        return s
    parts = _parts(c, s["pool"])
    for x in range(2):  # every page holds something, the places behind a sequence's last token too
        y = _normal(g, pages, h, page, d)
        if x == 0:
            y *= spread.unsqueeze(1)
        codes, scales = _quantise(y.half().float(), c["dtype"])
        parts[x].copy_(codes)
        parts[2 + x].copy_(scales)
    if c["op"] == "attention":
        s["q"] = (_normal(g, sum(n), c["heads"] * d) * (6.0 if c["softcap"] else 0.7)).half()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["c"] = case
    n, have = _lengths(case)
    s["total"], s["most"] = sum(n), (max(n), max(have))
    if case["op"] == "read":
        shape = (sum(n), case["kv_heads"] * case["head_dim"])
        s["k"], s["v"] = (torch.empty(shape, device=DEV, dtype=torch.float16) for _ in range(2))
    if case["op"] == "attention":
        s["o"] = torch.empty(sum(n), case["heads"] * case["head_dim"], device=DEV,
                             dtype=torch.uint8 if case["out"] == "e4m3" else torch.float16)
    if own:
        _prepare_own(s, case)
    return s


# ---------------------------------------------------------------- the library's calls

def _prepare_own(s, c):
    """What a program that calls the library keeps: the cache's and the batch's descriptions, options, workspace."""
    import vision_transformer_gb300 as vt

    dtype = vt.SV_DT_E4M3 if c["dtype"] == "e4m3" else vt.SV_DT_F16
    s["cache"] = vt.sv_cache(s["pool"], s["pool"].shape[0], c["page"], c["kv_heads"], c["head_dim"], dtype)
    s["batch"] = vt.sv_cache_batch(c["seqs"], s["table"], s["table"].stride(0), s["lengths"], s["prefix_pages"],
                                   c["prefix"])
    if c["op"] != "attention":
        s["stored"] = _stored(s)  # the pages' contents, which a call changes in place
        return
    s["options"] = vt.sv_attention_options(softcap=c["softcap"], mask=0 if c["mask"] == "document" else 1)
    size = vt.sv_attention_cached_workspace(s["cache"], s["batch"], s["total"], c["heads"])
    s["workspace"] = torch.zeros(size, device=DEV, dtype=torch.uint8)


def _run_own(s):
    import vision_transformer_gb300 as vt

    c = s["c"]
    if c["op"] == "write":
        vt.sv_cache_write(s["cache"], s["batch"], s["k"], s["v"], s["offsets"], s["total"],
                          k_stride=s["k"].stride(0), v_stride=s["v"].stride(0))
        return s["stored"]
    if c["op"] == "read":
        vt.sv_cache_read(s["cache"], s["batch"], s["k"], s["v"], s["offsets"], s["total"])
        return s["k"], s["v"]
    vt.sv_attention_cached(s["cache"], s["batch"], s["q"], s["o"], s["offsets"], s["total"], c["heads"],
                           options=s["options"], out_dtype=1 if c["out"] == "e4m3" else 0, workspace=s["workspace"])
    return s["o"].view(torch.float8_e4m3fn) if c["out"] == "e4m3" else s["o"]


# ---------------------------------------------------------------- plain forms

def _stored(s):
    """The cache's contents: numbers as they are stored, and their scales' bytes."""
    k, v, ke, ve = _parts(s["c"], s["pool"])
    as_type = torch.float8_e4m3fn if s["c"]["dtype"] == "e4m3" else torch.float16
    return {"k": k.view(as_type), "v": v.view(as_type), "k_scale": ke, "v_scale": ve}


def _values(c, codes, scales):
    """Stored numbers in 32 bits."""
    x = codes.contiguous().view(torch.float8_e4m3fn if c["dtype"] == "e4m3" else torch.float16).float()
    return x * torch.exp2(scales.float() - 16.0).unsqueeze(-1)


def _tokens(s, prefix):
    """Sequence of every token of the call, and its place: the number of its page in the pool and in the page."""
    c = s["c"]
    t = torch.arange(s["total"], device=DEV)
    off = s["offsets"].long()
    seq = torch.searchsorted(off[1:], t, right=True)
    pos = s["lengths"].long()[seq] - off[seq + 1] + t  # in the sequence's own tokens
    page = s["table"][seq, pos.clamp_min(0) // c["page"]].long()
    if prefix:
        first = pos < 0
        pos = torch.where(first, pos + prefix, pos)
        page = torch.where(first, s["prefix_pages"].long()[(pos // c["page"]).clamp_max(len(s["prefix_pages"]) - 1)], page)
    return page, pos % c["page"]


def _run_plain(s):
    c = s["c"]
    h, d = c["kv_heads"], c["head_dim"]
    parts = _parts(c, s["pool"])
    if c["op"] == "write":
        page, at = _tokens(s, 0)
        for x in range(2):
            codes, scales = _quantise(s["kv"[x]].float().reshape(-1, h, d), c["dtype"])
            parts[x][page, :, at] = codes
            parts[2 + x][page, :, at] = scales
        return _stored(s)
    if c["op"] == "read":
        page, at = _tokens(s, c["prefix"])
        for x in range(2):
            s["kv"[x]].copy_(_values(c, parts[x][page, :, at], parts[2 + x][page, :, at]).reshape(-1, h * d))
        return s["k"], s["v"]
    # queries padded to the longest: [seqs, kv_heads, group x queries, head_dim]
    group, (mq, mk) = c["heads"] // h, s["most"]
    off, have = s["offsets"].long(), s["lengths"].long()
    n = off[1:] - off[:-1]
    i = torch.arange(mq, device=DEV)
    real = i < n[:, None]
    q = s["q"][(off[:-1, None] + i) * real].float().view(-1, mq, h, group, d).permute(0, 2, 3, 1, 4)
    q = q.reshape(-1, h, group * mq, d) * (1.0 / math.sqrt(d))

    def gather(x, pages):  # [..., pages] -> [..., heads, tokens, head_dim] in 32 bits
        y = _values(c, parts[x][pages], parts[2 + x][pages])
        return y.transpose(-4, -3).flatten(-3, -2)

    table = s["table"].long().clamp_min(0)
    k, v = gather(0, table), gather(1, table)
    j = torch.arange(k.shape[2], device=DEV)
    limit = have[:, None].expand(-1, mq)
    if c["mask"] == "prefix":
        limit = torch.minimum(limit, i + (have - n + 1)[:, None]).clamp_min(0)
    hidden = (j >= limit[:, :, None]).unsqueeze(1).unsqueeze(1).expand(-1, -1, group, -1, -1).flatten(2, 3)
    p = torch.matmul(q, k.transpose(-1, -2))
    if c["softcap"]:
        p = p.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    p = p.masked_fill_(hidden, -math.inf)
    if c["prefix"]:
        pages = s["prefix_pages"].long()
        first = torch.matmul(q.transpose(0, 1).reshape(h, -1, d), gather(0, pages)[:, :c["prefix"]].transpose(-1, -2))
        if c["softcap"]:
            first = first.div_(c["softcap"]).tanh_().mul_(c["softcap"])
        first = first.view(h, -1, group * mq, c["prefix"]).transpose(0, 1)
        top = torch.maximum(p.amax(-1, keepdim=True), first.amax(-1, keepdim=True))
        first, p = torch.exp(first - top), p.sub_(top).exp_()
        o = torch.matmul(first.transpose(0, 1).reshape(h, -1, c["prefix"]), gather(1, pages)[:, :c["prefix"]])
        o = o.view(h, -1, group * mq, d).transpose(0, 1) + torch.matmul(p, v)
        o = o / (p.sum(-1, keepdim=True) + first.sum(-1, keepdim=True))
    else:
        p = p.sub_(p.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = o.view(-1, h, group, mq, d).permute(0, 3, 1, 2, 4)[real].reshape(-1, c["heads"] * d)
    if c["out"] == "e4m3":  # codes of 16 times the value
        return (o * 16.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    s["o"].copy_(o)
    return s["o"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    n, have = _lengths(c)
    h, d, page = c["kv_heads"], c["head_dim"], c["page"]
    codes, scales, _ = _layout(c)
    narrow = c["dtype"] == "e4m3"
    raw = s["pool"]

    def numbers(x):
        """All keys or values of the cache [pages, heads, page, head_dim]."""
        y = raw[:, x * codes:(x + 1) * codes].contiguous().view(torch.float8_e4m3fn if narrow else torch.float16)
        e = raw[:, 2 * codes + x * scales:2 * codes + (x + 1) * scales].double()
        return y.double().view(-1, h, page, d) * torch.pow(2.0, e.view(-1, h, page, 1) - 16.0)

    def sequence(x, i, all_numbers, prefix):
        """[tokens, heads, head_dim] of sequence i, behind the prefix where asked for."""
        own_pages = s["table"][i, :-(-have[i] // page)].long()
        y = all_numbers[own_pages].transpose(1, 2).reshape(-1, h, d)[:have[i]]
        if prefix and c["prefix"]:
            first = all_numbers[s["prefix_pages"].long()].transpose(1, 2).reshape(-1, h, d)[:c["prefix"]]
            y = torch.cat((first, y))
        return y

    if c["op"] == "write":
        out = {}
        for x, name in enumerate("kv"):
            to = torch.zeros(raw.shape[0], h, page, d, device=DEV, dtype=torch.float64)
            row = 0
            for i in range(c["seqs"]):
                y = s[name][row:row + n[i]].double().view(-1, h, d)
                row += n[i]
                if narrow:
                    least = torch.log2(y.abs().amax(-1, keepdim=True) / 448.0).clamp_min(-15.0)
                    # (magnitudes of 11 bits: what is 448 * 2^e up to 1e-6 is that)
                    y = y / torch.pow(2.0, torch.ceil(least - 1e-6))
                pos = torch.arange(have[i] - n[i], have[i], device=DEV)
                to[s["table"][i].long()[pos // page], :, pos % page] = y
            out[name] = to
        return out
    keys, values = numbers(0), numbers(1)
    if c["op"] == "read":
        return tuple(torch.cat([sequence(x, i, y, True)[-n[i]:] for i in range(c["seqs"])]).reshape(-1, h * d)
                     for x, y in enumerate((keys, values)))
    group = c["heads"] // h
    rows = []
    first = [y[s["prefix_pages"].long()].transpose(1, 2).reshape(-1, h, d)[:c["prefix"]] for y in (keys, values)] if c["prefix"] else None
    row = 0
    for i in range(c["seqs"]):
        k, v = sequence(0, i, keys, False), sequence(1, i, values, False)
        if first:
            k, v = torch.cat((first[0], k)), torch.cat((first[1], v))
        q = s["q"][row:row + n[i]].double().view(n[i], h, group, d)
        row += n[i]
        x = torch.einsum("nhgd,khd->hgnk", q, k) / math.sqrt(d)
        if c["softcap"]:
            x = c["softcap"] * torch.tanh(x / c["softcap"])
        if c["mask"] == "prefix":
            last = len(k) - n[i] + torch.arange(n[i], device=DEV)
            last = last.clamp_min(c["prefix"] - 1)  # every query sees the prefix
            x = torch.where(torch.arange(len(k), device=DEV) <= last[:, None], x, torch.full_like(x, -math.inf))
        p = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
        rows.append(torch.einsum("hgnk,khd->nhgd", p, v).reshape(n[i], -1))
    o = torch.cat(rows)
    return o * 16.0 if c["out"] == "e4m3" else o
