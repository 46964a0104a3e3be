"""What sv_rope and sv_qk_norm_rope do to the values of a head behind its rotated part."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

# (head_dim, rotated): runs of four, two and one pairs, runs of neighbouring pairs that the rotated part cuts
PARTS = [(128, 64), (72, 64), (24, 20), (80, 12), (40, 6), (16, 2), (256, 36), (96, 48)]


def _x(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).half().cuda()


def _bits(x):
    return x.contiguous().view(torch.int16)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("D,rot", PARTS)
def test_the_rest_of_a_head_is_left_as_it_is(sv, layout, in_place, D, rot):
    """Bit by bit: zeros of either sign, infinities, NaN of any payload beside ordinary values."""
    rows, heads = 37, 5
    x = _x(D + rot, rows, heads, D)
    pos = torch.randint(-3000, 3000, (1, rows), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    plan = sv.sv_rope_plan_init(rot, 1, layout)
    want = torch.empty_like(x)
    sv.sv_rope(x, want, pos, plan, rows, heads, D)
    special = torch.tensor([0x8000, 0x7C00, 0xFC00, 0x7E00, 0xFE55, 0x7C01, 0x0000, 0x0001], dtype=torch.int32)
    special = special.to(torch.int16).cuda()
    rest = _bits(x).view(rows, heads, D)[..., rot:]
    at = torch.randint(0, 16, rest.shape, generator=torch.Generator().manual_seed(2)).cuda()
    rest.copy_(torch.where(at < 8, special[at.clamp(max=7)], rest))
    before = _bits(x).clone().view(rows, heads, D)
    y = x if in_place else torch.empty_like(x)
    sv.sv_rope(x, y, pos, plan, rows, heads, D)
    sv.sv_sync()
    assert torch.equal(_bits(y).view(rows, heads, D)[..., rot:], before[..., rot:])
    assert torch.equal(y[..., :rot], want[..., :rot])


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("D,rot", PARTS + [(72, None), (128, None)])
def test_normalised_values_behind_the_rotated_part_stand_alone(sv, layout, D, rot):
    """An infinite value makes the RMS of its head infinite: the values that are not rotated become zeros, but for the
    infinite one, inf / inf. An infinite weight reaches its own value alone."""
    rows, heads = 9, 3
    x = _x(D, rows, heads, D)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")[None].contiguous()
    plan = sv.sv_rope_plan_init(rot, 1, layout) if rot else None
    keys = torch.zeros_like(x)
    y, z, want = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    gamma = _x(3, D)

    def call(q, out, g):
        sv.sv_qk_norm_rope(q, keys, out, z, g, None, pos if rot else None, plan, rows, heads, heads, D)
        sv.sv_sync()

    call(x, want, gamma)
    for at in (rot or 0, D - 1, (D + (rot or 0)) // 2):
        q = x.clone()
        q[4, 1, at] = math.inf
        call(q, y, gamma)
        head = y[4, 1, rot or 0:].clone()
        assert torch.isnan(head[at - (rot or 0)])
        head[at - (rot or 0)] = 0
        assert (head == 0).all(), at
        keep = torch.ones(rows, heads, dtype=torch.bool, device="cuda")
        keep[4, 1] = False
        assert torch.equal(y[keep], want[keep])
        g = gamma.clone()
        g[at] = math.nan
        call(x, y, g)
        rest = torch.arange(D, device="cuda") != at
        assert torch.equal(y[..., rest], want[..., rest]) and torch.isnan(y[..., at]).all()
