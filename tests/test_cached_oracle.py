"""The cache oracle against independent statements of the same: torch's e4m3 cast, brute force over
the int8 codes, a softmax written out."""
import math

import numpy as np
import pytest
import torch

from oracle import cached as C


def _bf16(rng, shape, spread=1.0):
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    return torch.as_tensor(x).bfloat16().double().numpy()


def test_e4m3_values_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    np.testing.assert_array_equal(C.e4m3_values(), codes.double().numpy())


@pytest.mark.parametrize("seed", range(4))
def test_e4m3_heads(seed):
    rng = np.random.default_rng(seed)
    for x in _bf16(rng, (50, 64), 3.0):
        codes, s = C.quantise_head(x, "e4m3")
        top = np.abs(x).max()
        assert math.frexp(s)[0] == 0.5 and 224 * s < top <= 448 * s
        want = torch.as_tensor(x / s).to(torch.float8_e4m3fn).double().numpy()
        np.testing.assert_array_equal(codes, want)


def test_e4m3_ties_and_ends():
    # top 448 gives scale 1; half ways: 17 -> 16 (even), 19 -> 20, and below the normal range
    x = np.array([448.0, 17, 19, -17, -19, 2.0 ** -10, 3 * 2.0 ** -10, 0])
    codes, s = C.quantise_head(x, "e4m3")
    assert s == 1
    np.testing.assert_array_equal(codes, [448, 16, 20, -16, -20, 0, 2 * 2.0 ** -9, 0])
    assert C.quantise_head([450.0] + [0.0] * 3, "e4m3")[1] == 2


@pytest.mark.parametrize("seed", range(3))
def test_int8_heads(seed):
    rng = np.random.default_rng(seed)
    grid = np.arange(-127, 128)
    for x in _bf16(rng, (30, 64)):
        codes, s = C.quantise_head(x, "int8")
        top = np.abs(x).max()
        far = np.abs(x[:, None] * 127 / top - grid)
        np.testing.assert_allclose(np.abs(x * 127 / top - codes), far.min(1), atol=1e-12)
        assert s == float(np.float32(top) / np.float32(127))
    # ties: 127 x / top = 0.5 and 1.5
    np.testing.assert_array_equal(C.quantise_head(np.array([254.0, 1, 3, -1, -3]), "int8")[0],
                                  [127, 0, 2, 0, -2])


def test_special_heads():
    for kind in ("int8", "e4m3"):
        codes, s = C.quantise_head(np.zeros(8), kind)
        assert s == 0 and not codes.any()
        for bad in (math.inf, math.nan):
            codes, s = C.quantise_head(np.array([1.0, bad]), kind)
            assert math.isnan(s) and not codes.any()


def test_places_of_ragged_rows():
    table = [[5, 2], [7, 9], [1, 3]]
    got = C.places(table, [17, 2, 0], [0, 3, 4, 5], 16, 9)
    assert got == [(0, 0, 14, 5, 14), (1, 0, 15, 5, 15), (2, 0, 16, 2, 0), (3, 1, 1, 7, 1)]


def test_attention_by_hand():
    rng = np.random.default_rng(0)
    k = [rng.standard_normal((6, 1, 4))]
    v = [rng.standard_normal((6, 1, 4))]
    q = rng.standard_normal((2, 2, 4))
    r = C.attention(q, k, v, [6], [0, 2], window=3, cap=5.0, slopes=[0.25, 0.0])
    for row, keys in ((0, (2, 3, 4)), (1, (3, 4, 5))):
        for h, slope in ((0, 0.25), (1, 0.0)):
            s = [5 * math.tanh(q[row, h] @ k[0][j, 0] / 2 / 5) - slope * (4 + row - j) for j in keys]
            w = np.exp(s)
            np.testing.assert_allclose(r["o"][row, h], w @ v[0][list(keys), 0] / w.sum())
            np.testing.assert_allclose(r["lse"][h, row], math.log(w.sum()))
    # a span: the first row sees the second too, and the window's reach stays
    r = C.attention(q, k, v, [6], [0, 2], window=3, span=True)
    s = [q[0, 0] @ k[0][j, 0] / 2 for j in (2, 3, 4, 5)]
    np.testing.assert_allclose(r["lse"][0, 0], math.log(np.exp(s).sum()))
    # nothing to see
    r = C.attention(q, k, v, [6], [0, 2], window=0)
    assert (r["o"] == 0).all() and np.isneginf(r["lse"]).all()
