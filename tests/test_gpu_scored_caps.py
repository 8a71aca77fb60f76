"""Capped scores beside a bias that is not linear in the key (the diagonal block, plans with a
position track), caps far above the scores, and rows of very different scores in one tile, against
the fp64 oracle.  Tolerances are those of the scored tests: the caps change none of their terms."""
import numpy as np
import pytest
import torch

import context_attention_metadata_gb300 as M
import workloads as wl
from marble_testlib import device_tracks
from oracle import mask, scored
from test_gpu_scored import HALF, INF, SOFT, _check, _np, _qkvdo, _run, _slopes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["usual", "signed"])
@pytest.mark.parametrize("cap", [1e-30, 0.1, 200.0, 1e4, 1e6, 1e8, 1e30])
def test_extreme_caps_beside_a_bias(cap, kind):
    n = 512
    tr = wl.random_pack(np.random.default_rng(3), n, max_samples=2)
    q, k, v, do = _qkvdo(n, 2, 2, 64, 3)
    slopes = _slopes(2, kind)
    pl = M.Plan(*device_tracks(tr), INF, 2)
    m = mask.dense_mask(tr, INF)
    for fused in (False, True):
        _check(_run(pl, q, k, v, do, M.Score(cap, slopes), fused=fused), q, k, v, do, m, cap, slopes)


@pytest.mark.parametrize("cap", [5.0, 200.0, 1e4, 1e6, 1e30])
def test_large_caps_on_a_position_track(cap):
    samples = [[wl.Span("causal", 90), wl.Span("group", 130), wl.Span("causal", 41),
                wl.Span("group", 200), wl.Span("causal", 51)],
               [wl.Span("causal", 100), wl.Span("full", 156)]]
    tr = wl.tracks_from_samples(samples)
    n = len(tr["sample"])
    perm = M.layout_vision_groups(tr["sample"], tr["seg"])
    moved = {x: np.asarray(tr[x])[perm] for x in tr}
    moved["pos"] = perm.astype(np.int32)
    s, g, z = device_tracks(moved)
    pl = M.Plan(s, g, z, INF, 2, "ptrr_block", pos=torch.as_tensor(moved["pos"]).cuda())
    m = mask.dense_mask(moved, INF)
    for d, slopes in ((64, _slopes(4, "usual")), (128, _slopes(4, "signed"))):
        q, k, v, do = _qkvdo(n, 4, 2, d, 8)
        for fused in (False, True):
            _check(_run(pl, q, k, v, do, M.Score(cap, slopes), fused=fused), q, k, v, do, m, cap,
                   slopes, moved["pos"])


@pytest.mark.parametrize("kind", [None, "usual"])
@pytest.mark.parametrize("cap", [50.0, 3e3, 1e6, 1e12, 1e20])
def test_small_scores_beside_scores_at_the_cap(cap, kind):
    """One row of every 32, and with it every tile, has scores of up to eight caps; the scores of the
    other rows are of order one.  Those keep their accuracy whatever the cap.  The large rows' dO
    is 0, which keeps them out of dK and dV (above a cap of 1e6 their P is not tested: an LSE of
    that size is rounded to more than one)."""
    n, d = 512, 64
    tr = wl.tracks_from_samples([[wl.Span("causal", 300), wl.Span("full", 212)]])
    q, k, v, do = _qkvdo(n, 2, 1, d, 12)
    big = torch.arange(n, device="cuda") % 32 == 5
    top = (q.double().transpose(0, 1) @ k[:, 0].double().T).abs().max().item() / 8
    gain = torch.where(big, 8.0 * cap / top, torch.ones_like(big, dtype=torch.float64))
    q = (q.double() * gain[:, None, None]).bfloat16()
    do = torch.where(big[:, None, None], torch.zeros_like(do), do)
    x = (q.double().transpose(0, 1) @ k[:, 0].double().T).abs() / 8
    # every warp's tile holds a score beyond 0.875 caps, the other rows none near the cap
    if cap > 100:
        assert x[:, ~big].max() < 0.01 * cap
    assert (x[:, big].reshape(2, -1, n // 64, 64).amax(-1) > 0.9 * cap).all()
    slopes = _slopes(2, kind)
    pl = M.Plan(*device_tracks(tr), INF, 2)
    m = mask.dense_mask(tr, INF)
    ref = scored.attention(q, k, v, m, cap, None if slopes is None else _np(slopes), do=do, h=HALF)
    rows, soft = (~big).cpu().numpy(), SOFT / HALF
    for fused in (False, True):
        O, L, dq, dk, dv = (_np(t) for t in _run(pl, q, k, v, do, M.Score(cap, slopes), fused=fused))
        assert (np.abs(L - ref["LSE"])[:, rows] <= SOFT).all()
        lim = (1 + HALF) * ((1 + soft) * ref["bound"]["O"] + HALF * np.abs(ref["O"]))
        assert (np.abs(O - ref["O"]) <= lim)[rows].all()
        if cap > 1e6:
            continue
        for name, got, at in (("dq", dq, rows), ("dk", dk, slice(None)), ("dv", dv, slice(None))):
            lim = (1 + HALF) * (1 + 4 * soft) * ref["bound"][name] + 1e-6
            assert (np.abs(got - ref[name]) <= lim)[at].all(), name


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("limit", [0.45, 0.875])
@pytest.mark.parametrize("side", [-1, 1])
def test_both_sides_of_a_limit(limit, side, bias):
    """The largest |scale q.k| / cap of every tile lies just below or just above one of the limits
    between the ways to tanh (0.45 and 0.875)."""
    n, d = 512, 128
    tr = wl.tracks_from_samples([[wl.Span("causal", 200), wl.Span("full", 312)]])
    q, k, v, do = _qkvdo(n, 2, 1, d, 15)
    # the same pair of vectors in every tile, whose product is far above the others'
    both = (-1.0) ** (torch.arange(d, device="cuda") // 3)
    q[::32], k[::64] = 2.0 * both, 1.5 * both
    x = (q.double().transpose(0, 1) @ k[:, 0].double().T).abs() / d ** 0.5
    tops = x.reshape(2, n // 32, 32, n // 64, 64).amax((2, 4))
    cap = 384 / d ** 0.5 / (limit * (1 + side * 1e-3))
    y = tops / cap
    assert ((y < limit) if side < 0 else (y > limit)).all() and (y - limit).abs().max() < 2e-3
    slopes = _slopes(2, "usual") if bias else None
    pl = M.Plan(*device_tracks(tr), INF, 2)
    _check(_run(pl, q, k, v, do, M.Score(cap, slopes), fused=True), q, k, v, do,
           mask.dense_mask(tr, INF), cap, slopes)
