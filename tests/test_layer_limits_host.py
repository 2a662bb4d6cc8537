"""Page tables whose positions 32 bits cannot count are refused, before any
HIP call."""
import ctypes

import pytest

import microscaling_fp4_block_mx_amd as mx

A, B, C, D, E, F = (i << 40 for i in range(1, 7))


@pytest.mark.parametrize("page", [32, 64, 128, 256])
def test_room_of_a_page_table(page):
    cache = mx.MxKVCache(A, B, C, D, 10, 1, 64, page)

    def status(width):
        # without a table: the next check behind the shapes'
        batch = mx.MxKVBatch(None, E, F, 1, 1, width)
        both = (mx.mx_kv_append(E, F, mx.MX_BF16, 64, 64, ctypes.byref(cache), ctypes.byref(batch), None),
                mx.mx_kv_attention(E, 64, 1, ctypes.byref(cache), ctypes.byref(batch), 0, 1.0, F, None, 0, None))
        assert both[0] == both[1]
        return both[0]

    fits = (2 ** 31 - 2048) // page
    assert status(fits) == mx.MX_ERR_NULL
    # tiles of 128 tokens behind the last one would begin past 2^31
    for width in (fits + 1, (2 ** 31 - 1) // page, 2 ** 31 // page, 2 ** 31 - 1):
        assert status(width) == mx.MX_ERR_SHAPE
