"""The scored-attention oracle against the plain one and against differences, and the refusals of
the scored calls that need no GPU."""
import ctypes

import numpy as np
import pytest

import context_attention_metadata_gb300 as M
import workloads as wl
from oracle import attention, mask, scored

RNG = np.random.default_rng


def _pack(seed, n=128):
    rng = RNG(seed)
    tr = wl.random_pack(rng, n, max_samples=3)
    q, k, v, do = (rng.standard_normal((n, h, 8)) for h in (4, 2, 2, 4))
    return tr, q, k, v, do


def test_without_change_it_is_the_plain_oracle():
    tr, q, k, v, do = _pack(0)
    m = mask.dense_mask(tr, 40)
    a = scored.attention(q, k, v, m, do=do)
    dq, dk, dv, O, L = attention.backward(q, k, v, do, m)
    for x, y in ((a["O"], O), (a["LSE"], L), (a["dq"], dq), (a["dk"], dk), (a["dv"], dv)):
        np.testing.assert_allclose(x, y, atol=1e-12)


@pytest.mark.parametrize("cap,bias", [(1.5, False), (0.0, True), (2.0, True)])
def test_gradients_against_differences(cap, bias):
    tr, q, k, v, do = _pack(1)
    m = mask.dense_mask(tr, wl.WINDOW_INF)
    slopes = [0.5, 0.1, -0.02, 0.0] if bias else None
    pos = RNG(2).permutation(len(q))

    def loss(q_, k_, v_):
        return (do * scored.attention(q_, k_, v_, m, cap, slopes, pos)["O"]).sum()

    a = scored.attention(q, k, v, m, cap, slopes, pos, do=do)
    rng, h = RNG(3), 1e-5
    for i, name in enumerate(("dq", "dk", "dv")):
        for _ in range(3):
            x = [q, k, v]
            e = rng.standard_normal(x[i].shape)
            e /= np.linalg.norm(e)
            up, dn = list(x), list(x)
            up[i], dn[i] = x[i] + h * e, x[i] - h * e
            diff = (loss(*up) - loss(*dn)) / (2 * h)
            # h^2 times a third derivative of order 1, and rounding of the loss (100) over h
            assert abs(diff - (a[name] * e).sum()) < 1e-7


def test_rows_without_a_key():
    tr, q, k, v, do = _pack(4)
    m = mask.dense_mask(tr, 0)
    a = scored.attention(q, k, v, m, 2.0, [0.1] * 4, do=do)
    empty = ~m.any(1)
    assert empty.any()
    assert (a["O"][empty] == 0).all() and np.isneginf(a["LSE"][:, empty]).all()
    assert (a["dq"][empty] == 0).all() and all(np.isfinite(a[x]).all() for x in ("dk", "dv"))


def test_refusals_without_a_plan():
    from context_attention_metadata_gb300 import _build
    _build.build()
    L = M.lib()
    s = M._Score(30.0, None)
    qkv, st = M._QKV(), M._State()
    r = ctypes.byref
    assert L.marble_attn_fwd_fused_scored(None, r(qkv), r(s), r(st), None) == M.ERR_INVALID_ARG
    assert b"plan is null" in L.marble_last_error()
    assert L.marble_attn_steps_scored(None, r(qkv), r(s), 0, None, None, None, r(st), None) == \
        M.ERR_INVALID_ARG
    assert L.marble_attn_bwd_fused_scored(None, r(qkv), r(s), None, None, None, None, None, None,
                                          None) == M.ERR_INVALID_ARG
    assert L.marble_attn_bwd_steps_scored(None, r(qkv), r(s), None, None, None, 0, None, None,
                                          None, None, None, None) == M.ERR_INVALID_ARG
