"""The rotary oracle against the definition as complex numbers and against differences, the
frequency tables, and the refusals of the rotary calls that need no GPU."""
import ctypes

import numpy as np
import pytest

import context_attention_metadata_gb300 as M
from oracle import rope as R


@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
def test_oracle_is_a_complex_rotation(pairing):
    rng = np.random.default_rng(0)
    freq, axis = M.rope_frequencies((8, 4, 4), 100.0)
    pos = rng.integers(-50, 50, (3, 7))
    x = rng.standard_normal((7, 2, 64))
    y = R.forward(x, pos, freq, axis, pairing)
    a, b = R.pair_channels(32, pairing)
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * (pos[axis].T * freq))[:, None]
    np.testing.assert_allclose(y[..., a], z.real, atol=1e-12)
    np.testing.assert_allclose(y[..., b], z.imag, atol=1e-12)
    np.testing.assert_array_equal(y[..., 32:], x[..., 32:])


@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
@pytest.mark.parametrize("norm", [False, True])
def test_oracle_gradient_against_differences(pairing, norm):
    rng = np.random.default_rng(1)
    freq, axis = M.rope_frequencies((5, 3), 50.0, "axial")
    pos = rng.integers(0, 99, (2, 3))
    x, g = rng.standard_normal((3, 2, 32)), rng.standard_normal((3, 2, 32))
    w = 1 + 0.3 * rng.standard_normal(32) if norm else None

    def loss(x_, w_):
        return (g * R.forward(x_, pos, freq, axis, pairing, w_, 1e-3)).sum()

    dx, dw = R.backward(g, x, pos, freq, axis, pairing, w, 1e-3)
    # central differences: the error is h^2 times third derivatives of order 10, and rounding
    # of the loss (order 10) over h
    h = 1e-5
    for at in [(0, 0, 0), (1, 1, 9), (2, 0, 15), (2, 1, 31)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    if norm:
        for c in (0, 7, 16, 31):
            e = np.zeros(32)
            e[c] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[c]) < 1e-7
    else:
        assert dw is None


def test_frequency_tables():
    f, a = M.rope_frequencies((4,), 16.0)
    np.testing.assert_allclose(f, [1, 0.5, 0.25, 0.125])
    assert (a == 0).all() and a.dtype == np.int32
    for layout in ("interleaved", "axial"):
        np.testing.assert_array_equal(M.rope_frequencies((4,), 16.0, layout)[0], f)
    f, a = M.rope_frequencies((2, 1, 1), 16.0)
    np.testing.assert_allclose(f, [1, 0.5, 0.25, 0.125])
    np.testing.assert_array_equal(a, [0, 0, 1, 2])
    f, a = M.rope_frequencies((2, 1, 1), 16.0, "interleaved")
    np.testing.assert_allclose(f, [1, 0.5, 0.25, 0.125])
    np.testing.assert_array_equal(a, [0, 1, 2, 0])
    f, a = M.rope_frequencies((2, 1, 1), 16.0, "axial")
    np.testing.assert_allclose(f, [1, 0.25, 1, 1])
    np.testing.assert_array_equal(a, [0, 0, 1, 2])
    for bad in ((), (0,), (3, -1)):
        with pytest.raises(ValueError):
            M.rope_frequencies(bad)
    with pytest.raises(ValueError):
        M.rope_frequencies((2,), layout="spiral")
    with pytest.raises(ValueError):
        M.Rope([1.0, 0.5], [0])
    with pytest.raises(ValueError):
        M.Rope([1.0, 0.5], pairing="thirds")


@pytest.fixture(scope="module")
def libm():
    from context_attention_metadata_gb300 import _build
    _build.build()
    return M.lib()


def _call(libm, back=False, n=4, d=64, axes=1, rot=32, pairing=0, freq=None, axis=None, eps=1e-6,
          dst_d=None, dst_v=True, rope=True, hq=2, hkv=1):
    """A rotary call on host buffers, which it refuses in the end; the arguments before that."""
    f = np.full(max(rot // 2, 1), 0.5) if freq is None else np.asarray(freq, np.float64)
    a = np.zeros(len(f), np.int32) if axis is None else np.asarray(axis, np.int32)
    buf = np.zeros(65536, np.float32)
    at = (buf.ctypes.data + 15) // 16 * 16
    c = M._Rope(axes, rot, pairing, f.ctypes.data, a.ctypes.data, at, None, None, eps)
    src = M._Heads(at, at, at, 256, 128, 128, hq, hkv, d)
    dst = M._Heads(at, at, at if dst_v else None, 256, 128, 128, hq, hkv, dst_d or d)
    r = ctypes.byref(c) if rope else None
    if back:
        st = libm.marble_rope_bwd(None, n, r, None, ctypes.byref(src), ctypes.byref(dst), None,
                                  None, None, None)
    else:
        st = libm.marble_rope(None, n, r, ctypes.byref(src), ctypes.byref(dst), None)
    return st, libm.marble_last_error()


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,msg", [
    (dict(rope=False), b"non-null"),
    (dict(n=-1), b"n_tokens"),
    (dict(n=2**31 - 1), b"n_tokens"),
    (dict(d=96), b"64 or 128"),
    (dict(dst_d=128), b"differ"),
    (dict(dst_v=False), b"same tensors"),
    (dict(hq=0), b"hq and hkv"),
    (dict(hkv=0), b"hq and hkv"),
    (dict(axes=0), b"n_axes"),
    (dict(axes=9), b"n_axes"),
    (dict(rot=0), b"rot_dim"),
    (dict(rot=24), b"rot_dim"),
    (dict(rot=80), b"rot_dim"),
    (dict(pairing=2), b"pairing"),
    (dict(freq=[float("nan")] * 16), b"finite"),
    (dict(freq=[float("inf")] * 16), b"finite"),
    (dict(axis=[1] * 16), b"axis"),
    (dict(axis=[-1] * 16), b"axis"),
    (dict(eps=-1.0), b"eps"),
    (dict(eps=float("nan")), b"eps"),
    (dict(eps=float("inf")), b"eps"),
    (dict(), b"device memory"),  # host buffers
])
def test_refusals(libm, back, kw, msg):
    st, err = _call(libm, back, **kw)
    assert st == M.ERR_INVALID_ARG and msg in err, (kw, err)


def test_empty_call_is_fine(libm):
    assert _call(libm, n=0)[0] == M.OK
    assert _call(libm, back=True, n=0)[0] == M.OK
