"""Packed attention in 64 bits, from the formulas, key by key visible (test helper)."""
import math

import torch


def limits(mask, lq, lk, prefix):
    if mask == 0:
        return [lk] * lq
    return [max(0, min(lk, max(i + lk - lq + 1, prefix))) for i in range(lq)]


def document(q, k, v, mask=0, prefix=0, scale=None, softcap=0.0, slopes=None):
    """q [Lq, Hq, D], k and v [Lk, Hk, D] -> o [Lq, Hq, D] in 64 bits and what bounds its error: sum p |v| and the
    largest |score| terms. Only visible keys enter a row."""
    lq, hq, d = q.shape
    lk, hk, _ = k.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    o = torch.zeros(lq, hq, d, dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    delta = torch.zeros(lq, hq, 1, dtype=torch.float64, device=q.device)
    lim = torch.tensor(limits(mask, lq, lk, prefix), device=q.device)
    if lk == 0:
        return o, a, delta
    g = hq // hk
    kh, vh = k.repeat_interleave(g, 1).permute(1, 2, 0), v.repeat_interleave(g, 1).permute(1, 0, 2)
    s = torch.matmul(q.permute(1, 0, 2), kh) * scale
    terms = torch.matmul(q.abs().permute(1, 0, 2), kh.abs()) * scale
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    if slopes is not None:
        away = (torch.arange(lq, device=q.device)[:, None] + (lk - lq) - torch.arange(lk, device=q.device)).abs()
        bias = slopes.double()[:, None, None] * away
        s, terms = s - bias, terms + bias
    seen = torch.arange(lk, device=q.device) < lim[:, None]
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    p = torch.where((lim > 0)[:, None], torch.softmax(s, -1), torch.zeros_like(s))
    p = torch.where(lim[:, None] > 0, p, torch.zeros_like(p))
    o = torch.matmul(p, vh).permute(1, 0, 2)
    a = torch.matmul(p, vh.abs()).permute(1, 0, 2)
    terms = torch.where(seen, terms, torch.zeros_like(terms))
    return o, a, terms.amax(-1).t().unsqueeze(-1)


def bound(o, a, terms, lk, vmax, d, softcap=0.0, e4m3=False):
    """What a result may be off by: F16 probabilities (2^-11 of sum p |v|) and output (2^-11; E4M3 2^-4, and 2^-14
    below its normal range at scale 16), scores in F32 (d products summed: d 2^-24 of their terms at most, and the few
    operations behind them; the cap adds 2^-22 of itself for tanh), their effect on a softmax twice their error."""
    ds = (d + 8) * 2.0 ** -24 * terms + 2.0 ** -21 * softcap
    err = (2.0 ** -11 + 2.0 ** -18 + 2 * ds) * a + lk * 2.0 ** -33 * vmax
    if e4m3:
        return err * (1 + 2.0 ** -4) + 2.0 ** -4 * o.abs() + 2.0 ** -14
    return err * (1 + 2.0 ** -11) + 2.0 ** -11 * o.abs() + 2.0 ** -25
