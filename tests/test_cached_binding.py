"""Calls on the paged cache that the library refuses on the host, without a GPU."""
import ctypes

import numpy as np
import pytest

import context_attention_metadata_gb300 as M


@pytest.fixture(scope="module")
def libm():
    from context_attention_metadata_gb300 import _build
    _build.build()
    return M.lib()


def _args(**kw):
    host = np.zeros(4096, np.int32)
    at = host.ctypes.data + -host.ctypes.data % 16
    c = dict(type=0, hkv=2, d=64, page_tokens=16, n_pages=4, k=at, v=at, k_stride=2048,
             v_stride=2048, k_scale=None, v_scale=None, k_scale_stride=0, v_scale_stride=0)
    s = dict(n_seqs=2, table_pages=2, table=at, table_stride=2, lens=at, start=None, status=None)
    a = dict(q=at, q_stride=256, o=at, o_stride=256, lse=None, hq=4, scale=0.0, window=5, span=0,
             new_tokens=1, workspace=at)
    n = kw.pop("n", 2)
    for k, v in kw.items():
        d = next(d for d in (c, s, a) if k in d)
        d[k] = v
    return n, M._Cache(*c.values()), M._Seqs(*s.values()), M._AttnCached(*a.values()), host


CACHE = [
    (dict(type=3), b"cache type"), (dict(type=-1), b"cache type"),
    (dict(d=96), b"head dim"), (dict(hkv=0), b"hkv"), (dict(page_tokens=24), b"page_tokens"),
    (dict(page_tokens=0), b"page_tokens"), (dict(page_tokens=65552), b"page_tokens"),
    (dict(n_pages=0), b"n_pages"), (dict(n_pages=1 << 31), b"n_pages"),
    (dict(k_stride=2047), b"page stride"), (dict(v_stride=2052), b"page stride"),
    (dict(k_stride=1 << 40), b"page stride"),
    (dict(type=2, k_scale_stride=31, v_scale_stride=32), b"scales"),
    (dict(type=1, k_scale_stride=32, v_scale_stride=34), b"scales"),
    (dict(n_seqs=-1, n=-1), b"n_tokens"), (dict(n=1), b"one row a sequence"),
    (dict(table_pages=0), b"table_pages"), (dict(table_stride=1), b"table_pages"),
    (dict(), b"device memory"),
]


@pytest.mark.parametrize("kw,msg", CACHE)
def test_cache_and_sequences(libm, kw, msg):
    n, c, s, a, host = _args(**kw)
    h = M._Heads(None, s.lens, s.lens, 0, 128, 128, 0, c.hkv, c.d)
    b = ctypes.byref
    for call in (lambda: libm.marble_cache_write(None, n, b(c), b(s), b(h), None),
                 lambda: libm.marble_cache_read(None, n, b(c), b(s), b(h), None),
                 lambda: libm.marble_attn_cached(n, b(c), b(s), b(a), None, None)):
        assert call() == M.ERR_INVALID_ARG
        assert msg in libm.marble_last_error(), libm.marble_last_error()


def test_null_descriptors(libm):
    n, c, s, a, host = _args()
    b = ctypes.byref
    assert libm.marble_cache_write(None, 2, None, b(s), None, None) == M.ERR_INVALID_ARG
    assert libm.marble_cache_read(None, 2, b(c), None, None, None) == M.ERR_INVALID_ARG
    assert libm.marble_attn_cached(2, None, None, None, None, None) == M.ERR_INVALID_ARG


def test_python_classes_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        M.Cache(x, x)
    with pytest.raises(ValueError):
        M.Sequences(torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
