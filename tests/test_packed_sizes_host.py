"""The size limit of sv_attention_packed as its documentation states it (no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def vt():
    from vision_transformer_gb300 import build
    build.build()
    import vision_transformer_gb300 as vt
    vt.load()
    return vt


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 22, 33, 43, 64])
@pytest.mark.parametrize("kv_heads", [64, 1000])
def test_calls_on_either_side_of_the_limit(vt, group, kv_heads):
    """(total_q / (256 / group) + docs) * kv_heads below 2^30: taken as far as the sizes go (and then turned down for a
    misaligned pointer, on the host), above: not supported."""
    lib = vt.load()
    buf = (ctypes.c_uint8 * 4096)()
    p = (ctypes.addressof(buf) + 15) // 16 * 16
    if group * kv_heads > 65536:
        pytest.skip("more heads than one call takes")
    per = 256 // group
    items = (2 ** 30 - 1) // kv_heads  # total_q / per + docs at most

    def call(total_q, docs):
        return lib.sv_attention_packed(p + 8, p, p, p, p, p, docs, total_q, 4, group * kv_heads, kv_heads, 8, 0, 0, 0, 0,
                                       None, 0, None, 0, None)

    most = min((items - 3) * per + per - 1, 2 ** 31 - 1 - 4096)
    assert call(most, 3) == vt.SV_ERR_INVALID_ARG
    docs = items - most // per
    if docs <= 2 ** 24:
        assert call(most, docs) == vt.SV_ERR_INVALID_ARG
        assert call(most, docs + 1) == vt.SV_ERR_UNSUPPORTED
    if (items - 3) * per + per <= 2 ** 31 - 1 - 4096:
        assert call((items - 3) * per + per, 3) == vt.SV_ERR_UNSUPPORTED
