"""sv_rope and sv_qk_norm_rope against the formulas in 64 bits.

Tolerance: one rounding to F16 (2^-11 relative, 2^-25 below the normal range), and for each pair the F32 angle
(2^-24 of half a turn, so below 2^-22), cosine and sine (2 ulp: 2^-22) and products: below 2^-20 (|a| + |b|). With a norm,
sums of up to 256 values in F32 (below 2^-19 relative in the scale and, through the mean, 2^-18 of the largest
normalised value).
"""
import numpy as np
import pytest
import torch

import rope_ref

pytestmark = pytest.mark.gpu


def _x(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).half()


def _check(got, ref, size, extra=0.0):
    got = got.double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(got).all()
    bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2.0 ** -20 * size + extra
    err = np.abs(got - ref)
    assert (err <= bound).all(), (err - bound).max()


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rows,heads,D,rot,axes", [
    (1, 1, 8, 8, 1), (1, 8, 128, 128, 1), (37, 3, 64, 64, 1), (5, 2, 72, 72, 2), (9, 5, 72, 72, 1), (4, 2, 72, 64, 1),
    (7, 3, 256, 256, 1), (6, 1, 80, 12, 1), (6, 2, 40, 6, 1), (3, 2, 16, 2, 1), (11, 7, 96, 36, 2), (2, 1, 248, 248, 2),
    (300, 16, 128, 64, 1), (1031, 12, 64, 32, 1), (13, 200, 24, 20, 2)])
def test_rope(sv, layout, rows, heads, D, rot, axes):
    x = _x(rows + D, rows, heads * D)
    pos = torch.randint(-5000, 5000, (axes, rows), dtype=torch.int32, generator=torch.Generator().manual_seed(3))
    y = torch.full((rows, heads * D), float("nan"), dtype=torch.float16, device="cuda")
    sv.sv_rope(x.cuda(), y, pos.cuda(), sv.sv_rope_plan_init(rot, axes, layout), rows, heads, D)
    sv.sv_sync()
    ref, size = rope_ref.rotate(x.double().numpy().reshape(rows, heads, D), pos.numpy(), rot, axes, layout, 10000.0)
    _check(y, ref, size)


@pytest.mark.parametrize("scaling,factor,original", [(0, 1.0, 0), (1, 8.0, 0), (2, 4.0, 0), (3, 16.0, 8192)])
def test_rope_far_positions(sv, scaling, factor, original):
    """Positions up to 2^31 - 1: the plan's frequencies carry 2^-53 relative, 2^-24 of a turn at that distance."""
    pos = torch.tensor([[0, 1, -1, 131071, 1048575, -1048576, 16777217, 2147483647]], dtype=torch.int32)
    rows, heads, D = pos.shape[1], 4, 128
    x = _x(5, rows, heads * D)
    y = torch.empty(rows, heads * D, dtype=torch.float16, device="cuda")
    sv.sv_rope(x.cuda(), y, pos.cuda(), sv.sv_rope_plan_init(D, 1, 0, 500000.0, scaling, factor, original), rows,
               heads, D)
    sv.sv_sync()
    ref, size = rope_ref.rotate(x.double().numpy().reshape(rows, heads, D), pos.numpy(), D, 1, 0, 500000.0, scaling,
                                factor, original)
    # both sides hold frequencies to about 2^-51 relative; at 2^31 positions that is 2^-20 radians
    _check(y, ref, size, extra=2.0 ** -19 * size)


def test_rope_strides_in_place_and_neighbours(sv):
    """A strided view rotated in place; values between the rows stay."""
    rows, heads, D, stride = 50, 4, 72, 600
    x = _x(9, rows, stride)
    dev = x.cuda()
    pos = torch.arange(rows, dtype=torch.int32)[None]
    plan = sv.sv_rope_plan_init(72)
    view = dev[:, 8:]
    sv.sv_rope(view, view, pos.cuda(), plan, rows, heads, D, x_stride=stride, y_stride=stride)
    sv.sv_sync()
    part = x[:, 8:8 + heads * D].double().numpy().reshape(rows, heads, D)
    ref, size = rope_ref.rotate(part, pos.numpy(), 72, 1, 0, 10000.0)
    _check(dev[:, 8:8 + heads * D], ref, size)
    assert torch.equal(dev[:, :8].cpu(), x[:, :8]) and torch.equal(dev[:, 8 + heads * D:].cpu(), x[:, 8 + heads * D:])


@pytest.mark.parametrize("norm", [0, 1])
@pytest.mark.parametrize("rows,hq,hk,D,rot,axes,layout", [
    (1, 1, 1, 8, 8, 1, 0), (1, 32, 8, 128, 128, 1, 0), (40, 16, 16, 72, 72, 2, 0), (17, 6, 2, 64, 64, 1, 1),
    (5, 3, 1, 80, 20, 1, 0), (3, 5, 5, 200, 100, 2, 1), (9, 2, 1, 16, 6, 1, 0), (700, 12, 4, 96, 96, 1, 0),
    (23, 7, 7, 72, None, 1, 0), (31, 4, 2, 128, None, 1, 0)])
def test_qk_norm_rope(sv, norm, rows, hq, hk, D, rot, axes, layout):
    """From the columns of a fused projection; rot None: the norm alone."""
    width = (hq + 2 * hk) * D
    qkv = (_x(rows + D, rows, width) * 3 + 0.5).half()
    gq, gk = (_x(1, D) * 0.2 + 1).half(), (_x(2, D) * 0.2 + 1).half()
    pos = torch.randint(0, 3000, (axes, rows), dtype=torch.int32, generator=torch.Generator().manual_seed(4))
    plan = sv.sv_rope_plan_init(rot, axes, layout) if rot else None
    dev = qkv.cuda()
    qo = torch.full((rows, hq * D), float("nan"), dtype=torch.float16, device="cuda")
    ko = torch.full((rows, hk * D), float("nan"), dtype=torch.float16, device="cuda")
    sv.sv_qk_norm_rope(dev, dev[:, hq * D:], qo, ko, gq.cuda(), gk.cuda(), pos.cuda() if rot else None, plan, rows, hq,
                       hk, D, norm=norm, eps=1e-6, q_stride=width, k_stride=width)
    sv.sv_sync()
    assert torch.equal(dev.cpu(), qkv)
    full = qkv.double().numpy().reshape(rows, hq + 2 * hk, D)
    for got, x, g in ((qo, full[:, :hq], gq), (ko, full[:, hq:hq + hk], gk)):
        ref = rope_ref.head_norm(x, g.double().numpy(), norm, 1e-6)
        top = np.abs(ref).max()
        size = np.abs(ref)
        if rot:
            ref, size = rope_ref.rotate(ref, pos.numpy(), rot, axes, layout, 10000.0)
        _check(got, ref, size, extra=2.0 ** -18 * (size + top))
    # the same in place, and without gammas
    q_in, k_in = dev[:, :hq * D], dev[:, hq * D:]
    sv.sv_qk_norm_rope(q_in, k_in, q_in, k_in, gq.cuda(), gk.cuda(), pos.cuda() if rot else None, plan, rows, hq, hk,
                       D, norm=norm, q_stride=width, k_stride=width, q_out_stride=width, k_out_stride=width)
    sv.sv_sync()
    assert torch.equal(dev[:, :hq * D], qo) and torch.equal(dev[:, hq * D:(hq + hk) * D], ko)
    assert torch.equal(dev[:, (hq + hk) * D:].cpu(), qkv[:, (hq + hk) * D:])
    sv.sv_qk_norm_rope(qkv.cuda(), qkv.cuda()[:, hq * D:], qo, ko, None, None, None, None, rows, hq, hk, D, norm=norm,
                       q_stride=width, k_stride=width)
    sv.sv_sync()
    ref = rope_ref.head_norm(full[:, :hq], 1.0, norm, 1e-6)
    _check(qo, ref, np.abs(ref), extra=2.0 ** -18 * (np.abs(ref) + np.abs(ref).max()))


def test_norm_of_zeros_and_constants(sv):
    """A head of zeros stays zero (eps), a constant head has no variance."""
    x = torch.cat([torch.zeros(1, 64), torch.full((1, 64), 3.0)]).half().cuda()
    y, z = torch.empty_like(x), torch.empty_like(x)
    for norm in (0, 1):
        sv.sv_qk_norm_rope(x, x, y, z, None, None, None, None, 2, 1, 1, 64, norm=norm, eps=1e-6)
        sv.sv_sync()
        assert (y[0] == 0).all() and (y[1] == (1.0 if norm == 0 else 0.0)).all() and torch.equal(y, z)


def test_rope_on_another_stream_and_in_a_graph(sv):
    rows, heads, D = 64, 4, 64
    x = _x(11, rows, heads * D).cuda()
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")[None]
    plan = sv.sv_rope_plan_init(64)
    want = torch.empty_like(x)
    sv.sv_rope(x, want, pos, plan, rows, heads, D)
    sv.sv_sync()
    side, y = torch.cuda.Stream(), torch.zeros_like(x)
    side.wait_stream(torch.cuda.current_stream())
    sv.sv_rope(x, y, pos, plan, rows, heads, D, stream=side)
    sv.sv_sync(side)
    assert torch.equal(y, want)
    g, y2 = torch.cuda.CUDAGraph(), torch.zeros_like(x)
    with torch.cuda.graph(g):
        sv.sv_rope(x, y2, pos, plan, rows, heads, D)
    x.copy_(x.flip(0))
    sv.sv_rope(x, want, pos, plan, rows, heads, D)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, want)


def test_rows_far_behind_the_first(sv):
    """In place behind 2^31 values, the bits of a compact copy."""
    stride, n, heads, D = 65536, 36000, 3, 72
    wide = torch.empty(n * stride, dtype=torch.float16, device="cuda").view(n, stride)
    gen = torch.Generator("cuda").manual_seed(7)
    x = torch.randn(n, heads * D, generator=gen, device="cuda").half()
    pos = torch.stack([torch.arange(n) % 191, torch.arange(n) // 191]).int().cuda()
    plan = sv.sv_rope_plan_init(D, 2, 0, 100.0)
    part = wide[:, 512:512 + heads * D]
    for norm in (False, True):
        part.copy_(x)
        y = torch.empty_like(x)
        if norm:
            z, zk = x[:, :D].contiguous(), torch.empty(n, D, dtype=torch.float16, device="cuda")
            sv.sv_qk_norm_rope(x, z, y, zk, None, None, pos, plan, n, heads, 1, D)
            sv.sv_qk_norm_rope(part, z, part, zk, None, None, pos, plan, n, heads, 1, D, q_stride=stride,
                               q_out_stride=stride)
        else:
            sv.sv_rope(x, y, pos, plan, n, heads, D)
            sv.sv_rope(part, part, pos, plan, n, heads, D, x_stride=stride, y_stride=stride)
        sv.sv_sync()
        assert torch.equal(part, y)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D,rot,layout", [(72, 72, 0), (128, 64, 1), (24, 20, 0)])
def test_a_head_of_nan_stays_alone(sv, bad, D, rot, layout):
    """Heads beside a head of NaN or infinities keep their bits, with and without the norm."""
    rows, heads = 40, 9
    x = _x(3, rows, heads * D).cuda()
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")[None].contiguous()
    plan = sv.sv_rope_plan_init(rot, 1, layout)
    runs = []
    for spoiled in (False, True):
        q = x.clone()
        if spoiled:
            q.view(rows, heads, D)[5, 4] = bad
            q.view(rows, heads, D)[39, 0, 1] = bad
        y, a, b = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
        sv.sv_rope(q, y, pos, plan, rows, heads, D)
        sv.sv_qk_norm_rope(q, x, a, b, None, None, pos, plan, rows, heads, heads, D, norm=1)
        sv.sv_sync()
        runs.append([t.view(rows, heads, D).clone() for t in (y, a, b)])
    keep = torch.ones(rows, heads, dtype=torch.bool, device="cuda")
    keep[5, 4] = keep[39, 0] = False
    for clean, got in zip(*runs):
        assert torch.equal(clean[keep], got[keep])
    assert torch.equal(runs[0][2], runs[1][2]) and not torch.isfinite(runs[1][1][5, 4]).any()
