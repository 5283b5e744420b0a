"""Sizes at the ends of the decode-time operators' 32-bit indices are refused on
the host (no GPU needed: fake pointers are never read)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def mx():
    from microscaling_block_quantization_b200 import build
    build.build()
    import microscaling_block_quantization_b200 as m
    m.lib()
    return m


@pytest.mark.parametrize("page_size,pages", [((1 << 31) - 1, 1), ((1 << 31) - 64, 1), (1 << 30, 2)])
def test_table_of_more_tokens_than_tiles_can_index(mx, page_size, pages):
    """A tile's tokens are numbered past the last visible one."""
    assert page_size * pages >= (1 << 31) - 64
    P = C.c_void_p
    c = C.byref(mx.mx_kv_cache(4096, 4096, 4096, 4096, None, None, 1, page_size, 1, 64))
    assert mx.mx_attn_decode(mx.MXFP4, c, P(4096), 0, 64, 1, 1, P(4096), pages, pages, P(4096), 0.1, 0, 0, P(4096), 0, 64, None,
                             P(4096), 0, None) == -1
