"""Calls of the key/value cache at the ends of what their documentation allows,
refused on the host before a launch that cannot be made. No compute call is made:
the pointers are never dereferenced."""

import pytest

from tests.test_abi_decode_cpu import FAKE, INVALID, SHAPE, q  # noqa: F401

LAST = 2 ** 31 - 1


def attn(q, heads=8, q_heads=32, dim=128, page=8, width=4, scale=0.1, n_pages=10):
    return q.qwha_cache_attn(FAKE, 1, 1, q_heads, FAKE, FAKE, FAKE, heads, dim, 4, 1, n_pages,
                             page, FAKE, width, FAKE, scale, FAKE, FAKE, 1 << 62, None)


@pytest.mark.parametrize("heads,q_heads", [(64, 64), (128, 128), (4096, 4096), (64, 4096),
                                           (4096, 61440)])
def test_attn_launches_of_too_many_workgroups(q, heads, q_heads):
    width = LAST // 8
    assert attn(q, heads=heads, q_heads=q_heads, width=width) == SHAPE
    assert b"workgroups" in q.qwha_last_error()
    assert q.qwha_cache_attn_workspace_bytes(1, q_heads, heads, 128, width, 8) == 0


def test_the_widest_table_of_few_heads_is_taken(q):
    assert q.qwha_cache_attn_workspace_bytes(1, 63, 63, 128, LAST // 8, 8) > 0
    assert q.qwha_cache_attn_workspace_bytes(1, 65528, 1, 128, LAST // 1024, 1024) > 0


@pytest.mark.parametrize("heads,dim", [(4, 256), (4096, 256), (16, 128)])
def test_rows_of_too_many_threads(q, heads, dim):
    T = LAST // (2 * heads)
    args = (heads, dim, 4, 1)
    assert q.qwha_cache_write(FAKE, FAKE, 1, T, FAKE, *args, 10, 16, FAKE, FAKE, FAKE,
                              None) == SHAPE
    assert q.qwha_cache_read(FAKE, FAKE, FAKE, *args, 10, 16, FAKE, T, 1, FAKE, FAKE,
                             None) == SHAPE


@pytest.mark.parametrize("scale", [3.0e38, -2.4e38, 3.4028234e38])
def test_scales_whose_powers_of_two_pass_fp32(q, scale):
    assert attn(q, scale=scale) == INVALID


def test_workspace_queries_out_of_range(q):
    layer = q.qwha_layer_decode_workspace_bytes
    assert layer(20, 256, 64, 500) > 0 and layer(64, 16384, 1 << 20, LAST) > 0
    for d_in in (32, 100, 65, 16448, 1 << 30, LAST):
        assert layer(20, d_in, 64, 500) == 0, d_in
    for d_out in ((1 << 20) + 1, LAST):
        assert layer(20, 256, d_out, 500) == 0, d_out
    for p in (256 * 64 + 1, LAST + 1, 1 << 62):
        assert layer(20, 256, 64, p) == 0, p
    assert layer(20, 16384, 1 << 20, LAST + 1) == 0
    rows = q.qwha_cache_attn_workspace_bytes
    assert rows(1, 32, 8, 128, 1 << 16, 16) > 0
    for page in (0, 4, 9, 24, 1000, 2048):
        assert rows(1, 32, 8, 128, 1 << 16, page) == 0, page
