"""sv_attention_cached at the ends of its range: results at the end of F16's."""
import pytest
import torch

from test_gpu_cached_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,have,prefix", [([1], 32, 0), ([1], 0, 32), ([40], 128, 0), ([20], 0, 128), ([200], 0, 128)])
@pytest.mark.parametrize("sign", [1, -1])
def test_values_at_the_end_of_f16(sv, n, have, prefix, sign):
    """A mean of equal values is that value, and finite: its error is one of 2^-11, which the largest F16 has no room for.

    Scores 0 and -ln 2 less a little: probabilities 2^8 and 128.07 (their head), of which F16 keeps 128.125, 4.3e-4
    more than the sum below; 65504 (1 + 2.4e-4) would round to infinity."""
    c = Case(n, [have], 1, 1, 64, prefix=prefix, e4m3=False, seed=1)
    tokens = have + prefix
    keys = torch.zeros(tokens, 1, 64, device="cuda", dtype=torch.float16)
    keys[1:, 0, 0] = -1.0
    places = c.b.places(0, -prefix, have)
    c.b.pool.store(0, *places, keys)
    c.b.pool.store(1, *places, torch.full_like(keys, sign * 65504.0))
    c.q.zero_()
    c.q[:, 0] = 1.0
    o = c.run(sv, scale=0.6926).double() * sign
    sv.sv_sync()
    # the formula's result is 65504; 2^-11 of it below, and no number above
    assert (o <= 65504).all() and (o >= 65504 * (1 - 2.0 ** -10)).all()
