"""Heads on which the norms of sv_qk_norm_rope lose their bits first."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _norm(sv, x, norm, eps):
    rows, d = x.shape
    y, z = torch.empty_like(x), torch.empty_like(x)
    sv.sv_qk_norm_rope(x, x, y, z, None, None, None, None, rows, 1, 1, d, norm=norm, eps=eps)
    sv.sv_sync()
    assert torch.equal(y, z)
    return y


@pytest.mark.parametrize("d", range(8, 257, 8))
def test_constant_heads_have_no_variance(sv, d):
    """d values of 11 bits sum exactly, so their mean is the value and nothing is left, however large it is."""
    values = torch.tensor([1.0, 3.0, 1001.0, 9999.0, 37472.0, 43712.0, 52448.0, 65504.0, -65504.0, 6e-8]).half()
    x = values[:, None].expand(-1, d).contiguous().cuda()
    assert (_norm(sv, x, sv.SV_NORM_LAYER, 1e-6) == 0).all()


@pytest.mark.parametrize("d", [72, 104, 120, 128, 240])
@pytest.mark.parametrize("base", [100.0, 2049.0, 40000.0])
def test_heads_far_from_zero(sv, d, base):
    """A few steps of F16 around a large mean. The mean is rounded to F32 (2^-24 of it), and the deviations' root mean
    square divides that; 2^-11 for the output, 2^-18 of the largest value for the sums."""
    rng = np.random.default_rng(d)
    step = float(np.spacing(np.float16(base)))
    x = (base + step * rng.integers(-3, 4, (40, d))).astype(np.float16)
    y = _norm(sv, torch.from_numpy(x).cuda(), sv.SV_NORM_LAYER, 1e-6).double().cpu().numpy()
    w = x.astype(np.float64)
    w = w - w.mean(1, keepdims=True)
    std = np.sqrt((w * w).mean(1, keepdims=True) + 1e-6)
    ref = w / std
    tol = 2.0 ** -11 * abs(ref) + 2.0 ** -25 + 2.0 ** -18 * abs(ref).max() + 1.01 * 2.0 ** -24 * base / std
    assert (abs(y - ref) <= tol).all()


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1e-30, 1e-6])
@pytest.mark.parametrize("norm", [0, 1])
def test_heads_of_zeros_with_any_eps(sv, eps, norm):
    """0 / sqrt(eps) is 0 for the smallest eps; other heads do not notice one like that."""
    x = torch.zeros(3, 72, dtype=torch.float16, device="cuda")
    x[1] = torch.linspace(-2.0, 3.0, 72).half()
    y = _norm(sv, x, norm, eps)
    assert (y[0] == 0).all() and (y[2] == 0).all()
    w = x[1].double() - (x[1].double().mean() if norm else 0.0)
    ref = w / ((w * w).mean() + eps).sqrt()
    assert ((y[1].double() - ref).abs() <= 2.0 ** -11 * ref.abs() + 2.0 ** -25 + 2.0 ** -18 * ref.abs().max()).all()
