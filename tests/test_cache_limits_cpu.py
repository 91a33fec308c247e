"""Where the cache calls refuse a size: at the limits that bsc.h states, not below them.  A call whose sizes are taken is
refused for a missing pointer here, which is checked later."""
import ctypes

import pytest

from test_cache_cpu import FAKE, _pools, _strides, ops  # noqa: F401

NULL, UNSUPPORTED = 1, 4


@pytest.mark.parametrize("B,T,Hkv,want", [
    (1, 2 ** 31 - 1, 2, NULL),                 # B T Hkv = 2^32 in 2^29 warps
    (1, 2 ** 31 - 1, 7, NULL),
    (1, 2 ** 31 - 1, 8, UNSUPPORTED),          # 2^31 warps
    (2 ** 26 - 1, 16, 16, NULL),               # 2^31 - 32 warps
    (2 ** 26, 16, 16, UNSUPPORTED),
    (2 ** 26, 1, 15, NULL),
    (2 ** 26, 1, 16, UNSUPPORTED),
    (357913941, 1, 3, NULL),                   # 2 * 3 * B = 2^31 - 2
    (357913942, 1, 3, UNSUPPORTED),
    (2 ** 31 - 1, 2 ** 31 - 1, 1 << 20, UNSUPPORTED)])
def test_write_and_read_limits(ops, B, T, Hkv, want):  # noqa: F811
    for P, call in ((ops.CacheWriteParams, ops.lib.mx_cache_write), (ops.CacheReadParams, ops.lib.mx_cache_read)):
        p = P(cache=_pools(ops, Hkv=Hkv, num_pages=1), k=0, v=FAKE, B=B, T=T, dtype=0, page_table=FAKE, table_stride=32,
              max_pages=32, seq_lens=FAKE, dev_status=FAKE, **_strides("kv"))
        assert call(ctypes.byref(p), None) == want


@pytest.mark.parametrize("B,T,Hq,Hkv,max_pages,want", [
    (2 ** 25 - 1, 1, 8, 8, 1, NULL),           # a tile of 8 rows each: 2^31 - 64 rows
    (2 ** 25, 1, 8, 8, 1, UNSUPPORTED),
    (2 ** 25, 1, 8, 8, 0, UNSUPPORTED),
    (2 ** 24, 1, 64, 8, 1, NULL),              # the same tiles full
    (1, 2 ** 31 - 33, 1, 1, 1, NULL),          # 2^31 - 32 rows in tiles of 32
    (1, 2 ** 31 - 31, 1, 1, 1, UNSUPPORTED),   # a tile more
    (1, 2 ** 20, 2047, 1, 1, NULL),
    (1, 2 ** 20, 2048, 1, 1, UNSUPPORTED),
    (1, 2 ** 31 - 1, 2 ** 30, 1, 1, UNSUPPORTED),
    (31, 1, 8, 8, 1 << 26, NULL),              # 2^23 chunks of each unit
    (32, 1, 8, 8, 1 << 26, UNSUPPORTED),
    (16, 3, 24, 8, 1 << 26, NULL),             # 9 rows: one tile of 16
    (8, 4, 64, 8, 1 << 26, NULL),              # 32 rows: one of 32
    (8, 17, 16, 8, 1 << 26, NULL),             # 34 rows: two, 2^30 chunks
    (16, 17, 16, 8, 1 << 26, UNSUPPORTED)])
def test_attention_limits(ops, B, T, Hq, Hkv, max_pages, want):  # noqa: F811
    p = ops.CacheAttnParams(cache=_pools(ops, Hkv=Hkv, num_pages=1), q=0, o=FAKE, B=B, T=T, Hq=Hq, dtype=0, softmax_scale=0.1,
                            page_table=FAKE, table_stride=max_pages, max_pages=max_pages, seq_lens=FAKE, workspace=FAKE,
                            workspace_bytes=1 << 40, **_strides("qo"))
    assert ops.lib.mx_cache_attn(ctypes.byref(p), None) == want


def test_workspace_of_sizes_at_the_limit(ops):  # noqa: F811
    """Sizes that the call takes are told their workspace, and no others."""
    tokens = 1 << 14
    B = 2 ** 31 // 24 - 1
    assert ops.mx_cache_attn_workspace_bytes(B, 1, 3, 3, 128, tokens) == 2 * 456 * 8 * 129 * 4
    assert ops.mx_cache_attn_workspace_bytes(2 ** 31 // 24 + 1, 1, 3, 3, 128, tokens) == 0
    assert ops.mx_cache_attn_workspace_bytes(1 << 12, 1, 64, 8, 128) == 2 * 456 * 8 * 129 * 4      # any table
