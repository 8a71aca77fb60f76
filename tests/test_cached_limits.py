"""Sizes of a paged cache at the ends of what the descriptors hold, refused on the host without a
GPU."""
import ctypes

import pytest

import context_attention_metadata_gb300 as M
from test_cached_binding import _args, libm  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(n_pages=(1 << 31) - 2, k_stride=1 << 38, v_stride=1 << 38),   # 2^70 bytes
    dict(n_pages=(1 << 31) - 2, k_stride=(1 << 29) + 8),               # 2^61
    dict(n_pages=(1 << 22) + 1, v_stride=1 << 38),                     # just beyond 2^61
    dict(type=2, n_pages=1 << 30, k_scale_stride=32, v_scale_stride=1 << 37)])
def test_pages_beyond_any_address(libm, kw):  # noqa: F811
    """Their last byte is beyond 2^60: products of pages and strides would overflow."""
    n, c, s, a, host = _args(**kw)
    h = M._Heads(None, s.lens, s.lens, 0, 128, 128, 0, c.hkv, c.d)
    b = ctypes.byref
    for call in (lambda: libm.marble_cache_write(None, n, b(c), b(s), b(h), None),
                 lambda: libm.marble_cache_read(None, n, b(c), b(s), b(h), None),
                 lambda: libm.marble_attn_cached(n, b(c), b(s), b(a), None, None)):
        assert call() == M.ERR_INVALID_ARG
        assert b"2^60" in libm.marble_last_error(), libm.marble_last_error()
