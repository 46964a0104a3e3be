"""Sizes of sv_attention_cached at and behind its limits (no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def vt():
    from vision_transformer_gb300 import build
    build.build()
    import vision_transformer_gb300 as vt
    vt.load()
    return vt


@pytest.fixture
def p():
    buf = (ctypes.c_uint8 * 4096)()
    yield (ctypes.addressof(buf) + 127) // 128 * 128
    del buf


@pytest.mark.parametrize("heads", [1, 8])
@pytest.mark.parametrize("total,prefix", [(2 ** 26, 2 ** 21), (2 ** 26, 2 ** 22 + 128), (2 ** 26, 2 ** 30), (2 ** 25, 2 ** 24),
                                          (2 ** 24, 2 ** 29 + 1), (3 * 2 ** 24, 2 ** 31 - 8192)])
def test_prefix_steps_beyond_the_limit(vt, p, total, prefix, heads):
    """Steps of 128 keys times blocks of 256 rows from 2^30 on are refused, their products beyond 32 bits too."""
    assert -(-total // 256) * -(-prefix // 128) >= 2 ** 30
    cache = vt.sv_cache(p, 4, 16, heads, 8)
    batch = vt.sv_cache_batch(1, p, 1, p, p, prefix)
    total //= heads
    assert vt.sv_attention_cached_workspace(cache, batch, total, heads) == 0
    assert b"too many" in vt.load().sv_last_error()
    assert vt.load().sv_attention_cached(cache, batch, p, p, p, total, heads, 0, 0, None, 0, p, 1 << 40,
                                         None) == vt.SV_ERR_UNSUPPORTED


@pytest.mark.parametrize("total,prefix", [(2 ** 20, 2 ** 24), (2 ** 12, 2 ** 31 - 8192), (1, 2 ** 31 - 8192)])
def test_prefix_steps_within_the_limit(vt, p, total, prefix):
    cache = vt.sv_cache(p, 4, 16, 1, 8)
    assert vt.sv_attention_cached_workspace(cache, vt.sv_cache_batch(1, p, 1, p, p, prefix), total, 1) > 0


@pytest.mark.parametrize("count,total,heads,kv_heads,dim", [(16, 16, 32, 8, 128), (16, 128, 32, 8, 128), (1, 1, 1, 1, 8), (256, 2048, 8, 8, 128),
                                                            (7, 32, 28, 4, 72), (2, 1, 64, 1, 128)])
@pytest.mark.parametrize("prefix", [0, 1, 5000])
def test_workspace_of_few_rows(vt, p, count, total, heads, kv_heads, dim, prefix):
    """At most 32 rows a sequence on average: 5.1 MB and what a prefix adds; never less than the counters' 4096 bytes."""
    rows = total * heads // kv_heads
    assert rows <= 32 * count
    size = vt.sv_attention_cached_workspace(vt.sv_cache(p, 4, 16, kv_heads, dim), vt.sv_cache_batch(count, p, 3, p, p, prefix), total, heads)
    blocks = -(-rows // 256) * 256 * kv_heads
    assert 4096 <= size <= 5.1e6 + (21e6 + blocks * 4 * (dim + 2) if prefix else 0)
