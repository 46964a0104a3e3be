"""Cases for measuring the rotary-position, query/key-norm and packed-attention operators.

``run`` computes a case in plain torch operations, or, with ``own`` set, through the
library's entry points: ``sv_rope``, ``sv_qk_norm_rope`` and ``sv_attention_packed``.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
SCALINGS = {"none": 0, "linear": 1, "base": 2, "by_parts": 3}


# ---------------------------------------------------------------- cases

def _rope(name, rows, heads, head_dim, rot, layout, base, scaling, factor, original, far):
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "head_dim": head_dim, "rot": rot, "axes": 1,
            "layout": layout, "base": base, "scaling": scaling, "factor": factor, "original": original, "far": far}


def _qk(name, rows, heads, kv_heads, head_dim, rot, axes, layout, norm, base, scaling, factor, original, far):
    return {"name": name, "op": "qk_norm_rope", "rows": rows, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rot": rot, "axes": axes, "layout": layout, "norm": norm, "base": base,
            "scaling": scaling, "factor": factor, "original": original, "far": far}


def _attn(name, docs, q_min, q_max, k_min, k_max, mix, heads, kv_heads, head_dim, mask="document", prefix=0,
          softcap=0.0, slopes=False, out="f16", fused=False):
    """Documents with q_min..q_max queries and k_min..k_max keys (q_max 0: as many queries as keys), drawn from `mix`."""
    return {"name": name, "op": "attention", "docs": docs, "q_min": q_min, "q_max": q_max, "k_min": k_min,
            "k_max": k_max, "mix": mix, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "mask": mask,
            "prefix": prefix, "softcap": softcap, "slopes": slopes, "out": out, "fused": fused}


def listed():
    return [
        # one new token of each of 8 requests, far into a context stretched eightfold: a call's latency
        _rope("rope_step", 8, 8, 128, 128, "half", 500000.0, "by_parts", 8.0, 8192, 65536),
        # the keys of a long prompt, half of each head rotated, neighbouring pairs
        _rope("rope_keys", 16411, 8, 128, 64, "interleaved", 10000.0, "linear", 4.0, 0, 16411),
        # one 378 px image: 27 x 27 patches, two position axes, heads of 72
        _qk("qk_image", 729, 16, 16, 72, 72, 2, "half", "layer", 100.0, "none", 1.0, 0, 27),
        # a batch of 32 such images
        _qk("qk_batch", 32 * 729, 16, 16, 72, 72, 2, "half", "rms", 100.0, "none", 1.0, 0, 27),
        # a long prompt with shared key heads
        _qk("qk_prompt", 8191, 32, 8, 128, 128, 1, "half", "rms", 1000000.0, "base", 2.0, 0, 8191),
        # pooling: one probe query for each of 64 images of different sizes
        _attn("attn_pool", 64, 1, 1, 64, 1024, 11, 16, 16, 72),
        # a batch of equal images, as the encoder runs them, from the fused projection's output
        _attn("attn_images", 32, 0, 0, 729, 729, 1, 16, 16, 72, fused=True),
        # 48 images of different sizes packed into one sequence, output for an E4M3 projection
        _attn("attn_packed", 48, 0, 0, 50, 1024, 5, 16, 16, 72, out="e4m3", fused=True),
        # prompts whose image prefix is visible to every query, scores capped
        _attn("attn_prefix_cap", 6, 0, 0, 900, 2100, 7, 16, 4, 128, mask="prefix", prefix=729, softcap=30.0),
        # prompts with a bias that falls with distance
        _attn("attn_distance", 5, 0, 0, 700, 2500, 3, 12, 12, 64, mask="prefix", slopes=True, fused=True),
        # one long prompt
        _attn("attn_long", 1, 0, 0, 8192, 8192, 1, 32, 8, 128, mask="prefix", fused=True),
        # one new token of each of 16 requests over long caches
        _attn("attn_step", 16, 1, 1, 900, 32768, 9, 32, 8, 128, mask="prefix"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "qk_norm_rope", "attention", "attention"])
    head_dim = rng.choice([64, 72, 80, 96, 128])
    if op != "attention":
        axes = rng.choice([1, 2]) if op == "qk_norm_rope" else 1
        rot = head_dim if rng.random() < 0.6 else 16 * rng.randint(1, head_dim // 16)
        layout = rng.choice(["half", "interleaved"])
        scaling = rng.choice(list(SCALINGS)) if axes == 1 else "none"
        factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0])
        base = rng.choice([10000.0, 500000.0]) if axes == 1 else 100.0
        rows, far = _log(rng, 1, 16000), _log(rng, 100, 100000) if axes == 1 else 64
        group = rng.choice([1, 2, 4, 8])
        kv = rng.randint(1, 16 // group)
        if op == "rope":
            c = _rope("", rows, kv * group, head_dim, rot, layout, base, scaling, factor, 4096, far)
        else:
            c = _qk("", rows, kv * group, kv, head_dim, rot, axes, layout, rng.choice(["rms", "layer"]), base, scaling,
                    factor, 4096, far)
    else:
        group = rng.choice([1, 1, 2, 3, 4, 8])
        kv = rng.randint(1, 16 // group)
        mask, cap = rng.choice(["document", "prefix"]), rng.choice([0.0, 0.0, 30.0, 50.0])
        slopes, out = rng.random() < 0.3, rng.choice(["f16", "f16", "e4m3"])
        if rng.random() < 0.35:  # few queries over long caches
            k_max = _log(rng, 300, 32768)
            docs = _log(rng, 1, max(1, min(64, 500000 // k_max)))
            q = rng.choice([1, 1, 1, 2, 5])
            c = _attn("", docs, q, q, max(q, k_max // 9), k_max, rng.randint(0, 999), kv * group, kv, head_dim, mask, 0,
                      cap, slopes, out)
        else:
            k_max = _log(rng, 17, 4096)
            docs = _log(rng, 1, max(1, min(64, (1 << 25) // (k_max * k_max))))
            c = _attn("", docs, 0, 0, max(1, k_max // 5), k_max, rng.randint(0, 999), kv * group, kv, head_dim, mask,
                      rng.choice([0, k_max // 3]), cap, slopes, out, rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(c):
    """(queries, keys) of every document."""
    r = random.Random(c["mix"])
    k = [r.randint(c["k_min"], c["k_max"]) for _ in range(c["docs"])]
    q = [r.randint(c["q_min"], c["q_max"]) for _ in range(c["docs"])] if c["q_max"] else list(k)
    return q, k


def _limits(c, lq, lk):
    """How many keys query 0, 1, ... of a document sees."""
    if c["mask"] == "document":
        return [lk] * lq
    return [max(0, min(lk, max(i + lk - lq + 1, c["prefix"]))) for i in range(lq)]


def work(c):
    if c["op"] == "rope":
        n = c["rows"] * c["heads"] * c["head_dim"]
        return {"bytes": 4 * n + 4 * c["rows"] * c["axes"], "flops": 3 * c["rows"] * c["heads"] * c["rot"]}
    if c["op"] == "qk_norm_rope":
        n = c["rows"] * (c["heads"] + c["kv_heads"]) * c["head_dim"]
        return {"bytes": 4 * n + 4 * c["rows"] * c["axes"], "flops": 7 * n}
    lq, lk = _lengths(c)
    seen = sum(sum(_limits(c, a, b)) for a, b in zip(lq, lk))
    d = c["head_dim"]
    q, kv = sum(lq) * c["heads"] * d, sum(lk) * c["kv_heads"] * d
    return {"bytes": 2 * q + 4 * kv + (1 if c["out"] == "e4m3" else 2) * q, "flops": 4 * seen * c["heads"] * d}


# ---------------------------------------------------------------- inputs

def _inputs(c, seed):
    """The inputs of a case, made from the seed."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)

    d = c["head_dim"]
    if c["op"] != "attention":
        rows = c["rows"]
        pos = torch.randint(0, c["far"], (c["axes"], rows), generator=g, device=DEV, dtype=torch.int32)
        if c["op"] == "rope":
            return {"x": normal(rows, c["heads"] * d).half(), "pos": pos}
        hq, hk = c["heads"], c["kv_heads"]
        qkv = (normal(rows, (hq + 2 * hk) * d) * 1.5).half()  # the fused projection's output
        return {"q": qkv[:, :hq * d], "k": qkv[:, hq * d:(hq + hk) * d], "pos": pos,
                "q_gamma": (1.0 + 0.2 * normal(d)).half(), "k_gamma": (1.0 + 0.2 * normal(d)).half()}
    lq, lk = _lengths(c)
    hq, hk = c["heads"], c["kv_heads"]
    s = {}
    if c["fused"]:  # queries, keys and values side by side in one row
        qkv = normal(sum(lk), (hq + 2 * hk) * d).half()
        s["q"], s["k"], s["v"] = qkv[:, :hq * d], qkv[:, hq * d:(hq + hk) * d], qkv[:, (hq + hk) * d:]
    else:
        s["q"], s["k"], s["v"] = normal(sum(lq), hq * d).half(), normal(sum(lk), hk * d).half(), normal(sum(lk), hk * d).half()
    if c["softcap"]:
        s["q"].mul_(8.0)  # scores beyond the cap among them

    def offsets(n):
        return torch.tensor([0] + n, device=DEV).cumsum(0).to(torch.int32)

    s["q_off"], s["k_off"] = offsets(lq), offsets(lk)
    s["prefix"] = torch.full((c["docs"],), c["prefix"], device=DEV, dtype=torch.int32) if c["prefix"] else None
    s["slopes"] = torch.exp2(-8.0 * (1 + torch.arange(hq, device=DEV)) / hq).float() if c["slopes"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["c"] = case
    d = case["head_dim"]
    half = {"device": DEV, "dtype": torch.float16}
    if case["op"] == "rope":
        s["y"] = torch.empty(case["rows"], case["heads"] * d, **half)
    elif case["op"] == "qk_norm_rope":
        s["q_out"] = torch.empty(case["rows"], case["heads"] * d, **half)
        s["k_out"] = torch.empty(case["rows"], case["kv_heads"] * d, **half)
    else:
        lq, lk = _lengths(case)
        s["total"], s["most"] = (sum(lq), sum(lk)), (max(lq), max(lk))
        s["o"] = torch.empty(s["total"][0], case["heads"] * d, device=DEV,
                             dtype=torch.uint8 if case["out"] == "e4m3" else torch.float16)
    if own:
        _prepare_own(s, case)
    return s


# ---------------------------------------------------------------- the library's calls

def _prepare_own(s, c):
    """What a program that calls the library keeps: the rotation's plan, or the attention's options and workspace."""
    import vision_transformer_gb300 as vt

    if c["op"] != "attention":
        s["plan"] = vt.sv_rope_plan_init(c["rot"], c["axes"], 0 if c["layout"] == "half" else 1, c["base"],
                                         SCALINGS[c["scaling"]], c["factor"], c["original"])
        return
    s["options"] = vt.sv_attention_options(softcap=c["softcap"], mask=0 if c["mask"] == "document" else 1,
                                           prefix=s["prefix"], slopes=s["slopes"])
    n = vt.sv_attention_packed_workspace(c["docs"], s["total"][0], s["total"][1], c["heads"], c["kv_heads"],
                                         c["head_dim"])
    s["workspace"] = torch.zeros(n, device=DEV, dtype=torch.uint8)


def _run_own(s):
    import vision_transformer_gb300 as vt

    c = s["c"]
    d = c["head_dim"]
    if c["op"] == "rope":
        vt.sv_rope(s["x"], s["y"], s["pos"], s["plan"], c["rows"], c["heads"], d)
        return s["y"]
    if c["op"] == "qk_norm_rope":
        vt.sv_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["q_gamma"], s["k_gamma"], s["pos"], s["plan"],
                           c["rows"], c["heads"], c["kv_heads"], d, norm=0 if c["norm"] == "rms" else 1, eps=1e-6,
                           q_stride=s["q"].stride(0), k_stride=s["k"].stride(0))
        return s["q_out"], s["k_out"]
    vt.sv_attention_packed(s["q"], s["k"], s["v"], s["o"], s["q_off"], s["k_off"], c["docs"], s["total"][0],
                           s["total"][1], c["heads"], c["kv_heads"], d, q_stride=s["q"].stride(0),
                           k_stride=s["k"].stride(0), v_stride=s["v"].stride(0), options=s["options"],
                           out_dtype=1 if c["out"] == "e4m3" else 0, workspace=s["workspace"])
    return s["o"].view(torch.float8_e4m3fn) if c["out"] == "e4m3" else s["o"]


# ---------------------------------------------------------------- plain forms

def _frequencies(c):
    """Radians per position of every pair of one axis, and the gain on cos and sin."""
    n = c["rot"] // 2 // c["axes"]
    i = torch.arange(n, device=DEV, dtype=torch.float64)
    base, gain = c["base"], 1.0
    if c["scaling"] == "base":
        base = base * c["factor"] ** (n / (n - 1))
    f = base ** (-i / n)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "by_parts":
        ramp = ((c["original"] * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        f, gain = f * (ramp + (1 - ramp) / c["factor"]), 0.1 * math.log(c["factor"]) + 1
    return f, gain


def _rotate(x, pos, c):
    """x [rows, heads, head_dim] in 32 bits."""
    rows, heads, d = x.shape
    axes, rot = c["axes"], c["rot"]
    n = rot // 2 // axes
    f, gain = _frequencies(c)
    t = pos.t().double().unsqueeze(-1) * f  # [rows, axes, n]: far positions need 64 bits
    cos, sin = (t.cos() * gain).float().unsqueeze(1), (t.sin() * gain).float().unsqueeze(1)
    part = x[..., :rot].reshape(rows, heads, axes, 2, n) if c["layout"] == "half" else x[..., :rot].reshape(rows, heads, axes, n, 2).transpose(-1, -2)
    a, b = part[..., 0, :], part[..., 1, :]
    part = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-2)
    if c["layout"] != "half":
        part = part.transpose(-1, -2)
    return torch.cat((part.reshape(rows, heads, rot), x[..., rot:]), dim=-1)


def _norm(x, gamma, c):
    if c["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * gamma.float()


def _run_plain(s):
    c = s["c"]
    d = c["head_dim"]
    if c["op"] == "rope":
        s["y"].copy_(_rotate(s["x"].float().view(c["rows"], c["heads"], d), s["pos"], c).reshape(c["rows"], -1))
        return s["y"]
    if c["op"] == "qk_norm_rope":
        q = _norm(s["q"].float().reshape(c["rows"], c["heads"], d), s["q_gamma"], c)
        k = _norm(s["k"].float().reshape(c["rows"], c["kv_heads"], d), s["k_gamma"], c)
        s["q_out"].copy_(_rotate(q, s["pos"], c).reshape(c["rows"], -1))
        s["k_out"].copy_(_rotate(k, s["pos"], c).reshape(c["rows"], -1))
        return s["q_out"], s["k_out"]
    # every document padded to the longest: [docs, kv_heads, group, queries, keys]
    hq, hk = c["heads"], c["kv_heads"]
    mq, mk = s["most"]
    q0, k0 = s["q_off"][:-1].long(), s["k_off"][:-1].long()
    lq, lk = (s["q_off"][1:] - s["q_off"][:-1]).long(), (s["k_off"][1:] - s["k_off"][:-1]).long()
    i, j = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
    real_q, real_k = i < lq[:, None], j < lk[:, None]  # [docs, mq], [docs, mk]
    at_q, at_k = ((q0[:, None] + i) * real_q), ((k0[:, None] + j) * real_k)
    q = s["q"][at_q].float().view(-1, mq, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    k = s["k"][at_k].float().view(-1, mk, hk, d).permute(0, 2, 3, 1).unsqueeze(2)
    v = s["v"][at_k].float().view(-1, mk, hk, d).permute(0, 2, 1, 3).unsqueeze(2)
    at = i + (lk - lq)[:, None]  # position of each query among the keys
    limit = lk[:, None].expand(-1, mq)
    if c["mask"] == "prefix":
        limit = torch.minimum(limit, torch.clamp_min(at + 1, c["prefix"]))
    p = torch.matmul(q, k).mul_(1.0 / math.sqrt(d))
    if c["softcap"]:
        p = p.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    if c["slopes"]:
        p = p.sub_(s["slopes"].view(1, hk, hq // hk, 1, 1) * (at[:, :, None] - j).abs().float()[:, None, None])
    hidden = (j >= limit[:, :, None])[:, None, None]
    p = p.masked_fill_(hidden, -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = o.permute(0, 3, 1, 2, 4)[real_q].reshape(-1, hq * d)
    if c["out"] == "e4m3":  # codes of 16 times the value
        return (o * 16.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    s["o"].copy_(o)
    return s["o"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    c = case

    def turn(x, pos):
        """Rotation as a product of complex numbers, pair by pair."""
        rows, heads, d = x.shape
        per_axis = c["rot"] // c["axes"]
        n = per_axis // 2
        freqs = []
        for i in range(n):
            if c["scaling"] == "base":
                f = (c["base"] * c["factor"] ** (n / (n - 1))) ** (-i / n)
            else:
                f = c["base"] ** (-i / n)
            if c["scaling"] == "linear":
                f /= c["factor"]
            elif c["scaling"] == "by_parts":
                turns = c["original"] * f / (2 * math.pi)
                keep = min(1.0, max(0.0, (turns - 1.0) / 31.0))
                f = keep * f + (1.0 - keep) * f / c["factor"]
            freqs.append(f)
        gain = 1.0 + 0.1 * math.log(c["factor"]) if c["scaling"] == "by_parts" else 1.0
        y = x.clone()
        f = torch.tensor(freqs, device=x.device, dtype=torch.float64)
        for axis in range(c["axes"]):
            z = gain * torch.exp(1j * (pos[axis].double()[:, None] * f))  # [rows, n]
            lo = axis * per_axis
            if c["layout"] == "half":
                first, second = slice(lo, lo + n), slice(lo + n, lo + per_axis)
            else:
                first, second = slice(lo, lo + per_axis, 2), slice(lo + 1, lo + per_axis, 2)
            w = torch.complex(x[..., first], x[..., second]) * z[:, None, :]
            y[..., first], y[..., second] = w.real, w.imag
        return y

    s = _inputs(c, seed)
    d, hq = c["head_dim"], c["heads"]
    if c["op"] == "rope":
        return turn(s["x"].double().view(-1, hq, d), s["pos"]).reshape(c["rows"], -1)
    if c["op"] == "qk_norm_rope":
        got = []
        for x, gamma in ((s["q"], s["q_gamma"]), (s["k"], s["k_gamma"])):
            x = x.double().reshape(c["rows"], -1, d)
            if c["norm"] == "layer":
                x = x - x.sum(-1, keepdim=True) / d
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + 1e-6) * gamma.double()
            got.append(turn(x, s["pos"]).reshape(c["rows"], -1))
        return tuple(got)
    lq, lk = _lengths(c)
    group = hq // c["kv_heads"]
    out = torch.zeros(sum(lq), hq * d, device=DEV, dtype=torch.float64)
    q0 = k0 = 0
    for nq, nk in zip(lq, lk):
        limit = torch.tensor(_limits(c, nq, nk), device=DEV)
        keys = torch.arange(nk, device=DEV)
        away = (torch.arange(nq, device=DEV)[:, None] + (nk - nq) - keys[None, :]).abs().double()
        for h in range(hq):
            at = slice(h * d, h * d + d)
            kv = slice(h // group * d, h // group * d + d)
            x = s["q"][q0:q0 + nq, at].double() @ s["k"][k0:k0 + nk, kv].double().t() / math.sqrt(d)
            if c["softcap"]:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            if c["slopes"]:
                x = x - float(s["slopes"][h]) * away
            x = torch.where(keys[None, :] < limit[:, None], x, torch.full_like(x, -math.inf))
            p = torch.nan_to_num(torch.softmax(x, dim=-1), nan=0.0)  # a query that sees nothing: zero
            out[q0:q0 + nq, at] = p @ s["v"][k0:k0 + nk, kv].double()
        q0, k0 = q0 + nq, k0 + nk
    return out * 16.0 if c["out"] == "e4m3" else out
