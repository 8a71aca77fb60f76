"""Attention with capped scores and a bias by distance on the GPU against the fp64 oracle.

Tolerances.  P and dS are rounded to bf16 before their products, O before delta: half a step,
2^-8, each, carried to every result by the oracle's bounds; results are fp32 or rounded to bf16
once more.  The rest is fp32: a score of size S is off by 2^-24 times (d for the sum of d
products, 4 for cap and bias, both below 2^-22 of the scores' size), for |S| up to 40 and the sum
of |products| up to four times that 128 * 2^-24 * 160 = 1.2e-3 at the very worst, which changes a
weight by that factor; the root of d in place of d gives 1.1e-4, which is allowed here (SOFT) for
the LSE and, times the size of the terms, for everything else."""
import numpy as np
import pytest
import torch

import context_attention_metadata_gb300 as M
import workloads as wl
from marble_testlib import device_tracks, rel_fro
from oracle import mask, scored

pytestmark = pytest.mark.gpu
HALF = torch.finfo(torch.bfloat16).eps / 2
SOFT = 1.2e-4
INF = wl.WINDOW_INF


def _slopes(hq, kind):
    s = {None: None, "usual": [2.0 ** (-8 * (h + 1) / hq) for h in range(hq)],
         "signed": [(-1) ** h * 0.01 * (h + 1) for h in range(hq)],
         "steep": [3.0 + h for h in range(hq)], "zero": [0.0] * hq}[kind]
    return None if s is None else torch.tensor(s, dtype=torch.float32, device="cuda")


def _qkvdo(n, hq, hkv, d, seed, scale=1.5):
    q, k, v, do = wl.make_qkvdo(n, hq, hkv, d, device="cuda", seed=seed)
    return (q.float() * scale).bfloat16(), k, v, do


def _run(pl, q, k, v, do, score, needed=False, fused=False, merge="carried", stream=None):
    """Forward and backward, everything back in original order: O, LSE, dq, dk, dv."""
    n, hq, d = q.shape
    qp, kp, vp, dp = (pl.permute(x) for x in (q, k, v, do))
    st = M.State(n, hq, d)
    o, lse = torch.empty_like(qp), torch.empty((hq, n), device="cuda")
    delta = torch.empty_like(lse)
    dq, dk, dv = (torch.zeros(x.shape, device="cuda") for x in (q, k, v))
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    M.forward(pl, qp, kp, vp, st, o, lse, needed=needed, fused=fused, merge=merge, score=score,
              stream=stream)
    M.backward(pl, qp, kp, vp, o, dp, lse, delta, dq, dk, dv, needed=needed, fused=fused,
               score=score, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    pl.check()
    perm = pl.export("perm").long()
    out = torch.empty_like(lse)
    out[:, perm] = lse
    return (pl.permute(o, inverse=True), out) + tuple(pl.permute(x, inverse=True)
                                                      for x in (dq, dk, dv))


def _np(x):
    return x.double().cpu().numpy()


def _check(got, q, k, v, do, m, cap, slopes, pos=None, scale=None, steps=1):
    """steps: roundings of O to bf16 (one, or the bf16 merge's)."""
    ref = scored.attention(q, k, v, m, cap, None if slopes is None else _np(slopes), pos, scale,
                           do, HALF)
    b = ref["bound"]
    O, L = _np(got[0]), _np(got[1])
    soft = SOFT / HALF  # the bounds are HALF times the size of the terms
    # the rounding of P differs from the exact by half a step of the rounded value
    assert (np.abs(O - ref["O"]) <= (1 + HALF) * ((1 + soft) * b["O"] +
                                                  steps * HALF * np.abs(ref["O"]) + 1e-30)).all()
    live = np.isfinite(ref["LSE"])
    assert (np.isfinite(L) == live).all() and (L[~live] == -np.inf).all()
    assert (np.abs(L[live] - ref["LSE"][live]) <= SOFT).all()
    for name, x in zip(("dq", "dk", "dv"), got[2:]):
        err = np.abs(_np(x) - ref[name])
        # both dS and P carry the factor of the scores' error, and delta that of O
        assert (err <= (1 + HALF) * (1 + 4 * soft) * b[name] + 1e-6).all(), \
            (name, (err - b[name]).max())
        # over all entries the roundings average: the error's square is at most the sum of their
        # variances, each at most the square of half a step (a third of it, if evenly spread)
        assert np.linalg.norm(err) <= np.sqrt(ref["noise"][name].sum()) + 1e-6, name


MODES = [(30.0, None), (2.0, None), (0.0, "usual"), (5.0, "usual"), (1.0, "signed"),
         (0.0, "steep"), (0.0, "signed")]


@pytest.mark.parametrize("seed", range(14))
def test_random_packs(seed):
    cap, kind = MODES[seed % len(MODES)]
    rng = np.random.default_rng(4000 + seed)
    n = 128 * int(rng.choice([1, 2, 4, 8]))
    tr = wl.random_pack(rng, n, max_samples=int(rng.integers(1, 5)))
    d, hkv = int(rng.choice([64, 128])), int(rng.choice([1, 2, 3]))
    hq = hkv * int(rng.choice([1, 2, 4]))
    P = int(rng.choice([p for p in (1, 2, 4) if (n // 128) % p == 0]))
    W = int(rng.choice([INF, 1, 60, 300]))
    order = ["contiguous", "ptrr_block"][seed % 2]
    q, k, v, do = _qkvdo(n, hq, hkv, d, seed)
    slopes = _slopes(hq, kind)
    pl = M.Plan(*device_tracks(tr), W, P, order)
    m = mask.dense_mask(tr, W)
    score = M.Score(cap, slopes)
    for kw in ({}, {"needed": True}, {"fused": True}):
        _check(_run(pl, q, k, v, do, score, **kw), q, k, v, do, m, cap, slopes)


@pytest.mark.parametrize("cap,kind", [(2.0, "usual"), (20.0, None), (0.0, "signed")])
@pytest.mark.parametrize("cid", [1, 2, 5])
def test_small_configurations(cid, cap, kind):
    n = 2048
    tr = wl.config_tracks(cid, n)
    q, k, v, do = _qkvdo(n, 4, 2, 128, cid)
    slopes = _slopes(4, kind)
    pl = M.Plan(*device_tracks(tr), INF, 4, "ptrr_block")
    m = mask.dense_mask(tr, INF)
    for fused in (False, True):
        _check(_run(pl, q, k, v, do, M.Score(cap, slopes), fused=fused), q, k, v, do, m, cap, slopes)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_without_a_key(d):
    tr = wl.tracks_from_samples([[wl.Span("causal", 300), wl.Span("full", 200)],
                                 [wl.Span("causal", 12)]])
    q, k, v, do = _qkvdo(512, 2, 1, d, 5)
    slopes = _slopes(2, "usual")
    pl = M.Plan(*device_tracks(tr), 0, 2)
    m = mask.dense_mask(tr, 0)
    for fused in (False, True):
        got = _run(pl, q, k, v, do, M.Score(3.0, slopes), fused=fused)
        assert (got[0][:300] == 0).all() and (got[2][:300] == 0).all()
        _check(got, q, k, v, do, m, 3.0, slopes)


# Long rows on few heads, which the fused forward cuts into pieces: one long sample; an odd number
# of blocks; short samples, whose rows have fewer tiles than there are pieces, beside a long one;
# rows that see no key (window 0) beside a long bidirectional span
LONG = [
    ([[wl.Span("causal", 2048)]], INF, 4, 2, 1, 64, 2.0, "usual"),
    ([[wl.Span("causal", 2944)]], INF, 1, 1, 1, 128, 0.0, "steep"),
    ([[wl.Span("causal", 1900)]] + [[wl.Span("causal", 55), wl.Span("full", 45)]] * 6 +
     [[wl.Span("noise", 60)]], INF, 4, 2, 2, 64, 30.0, None),
    ([[wl.Span("causal", 300), wl.Span("full", 1700)], [wl.Span("causal", 48)]], 0, 2, 2, 1, 128, 3.0,
     "signed"),
]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_rows_in_pieces(case):
    samples, W, P, hq, hkv, d, cap, kind = LONG[case]
    tr = wl.tracks_from_samples(samples)
    pad = -len(tr["sample"]) % (128 * P)
    if pad:
        tr = wl.tracks_from_samples(samples + [[wl.Span("causal", pad)]])
    n = len(tr["sample"])
    q, k, v, do = _qkvdo(n, hq, hkv, d, 60 + case)
    slopes = _slopes(hq, kind)
    pl = M.Plan(*device_tracks(tr), W, P, "ptrr_block")
    score = M.Score(cap, slopes)
    M.timing_enable(True)
    M.timing_read()
    got = _run(pl, q, k, v, do, score, fused=True)
    launches = M.timing_read()["fwd_launches"]
    M.timing_enable(False)
    assert launches == 2  # the pieces and their join
    _check(got, q, k, v, do, mask.dense_mask(tr, W), cap, slopes)
    again = _run(pl, q, k, v, do, score, fused=True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_pieces_of_two_streams_at_once():
    """Two forwards of one plan on two streams, over and over: each has pieces of its own."""
    n = 2048
    tr = wl.tracks_from_samples([[wl.Span("causal", n)]])
    pl = M.Plan(*device_tracks(tr), INF, 1)
    runs = []
    for seed in (71, 72):
        q, k, v, _ = _qkvdo(n, 2, 1, 64, seed)
        runs.append((q, k, v, M.State(n, 2, 64), torch.empty_like(q),
                     torch.empty((2, n), device="cuda"), torch.cuda.Stream()))
    score = M.Score(5.0)
    want = []
    for q, k, v, st, o, lse, _ in runs:
        M.forward(pl, q, k, v, st, o, lse, fused=True, score=score)
        want.append((o.clone(), lse.clone()))
        o.zero_(), lse.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for q, k, v, st, o, lse, stream in runs:
            M.forward(pl, q, k, v, st, o, lse, fused=True, score=score, stream=stream)
    torch.cuda.synchronize()
    pl.check()
    for (q, k, v, st, o, lse, _), (a, b) in zip(runs, want):
        assert torch.equal(o, a) and torch.equal(lse, b)


def test_pieces_keep_nan_and_infinity():
    """A key's NaN or infinite value reaches the rows that see it, and no row of an earlier block
    (a masked key's weight is a zero of the product)."""
    n = 2048
    tr = wl.tracks_from_samples([[wl.Span("causal", n)]])
    q, k, v, _ = _qkvdo(n, 1, 1, 64, 70)
    pl = M.Plan(*device_tracks(tr), INF, 1)
    for key, bad in ((700, float("nan")), (5, float("inf")), (1500, float("-inf"))):
        x = v.clone()
        x[key, 0, 3] = bad
        st, o, lse = M.State(n, 1, 64), torch.empty_like(q), torch.empty((1, n), device="cuda")
        M.forward(pl, q, k, x, st, o, lse, fused=True, score=M.Score(5.0))
        pl.check()
        assert torch.isfinite(lse).all()
        hit = ~torch.isfinite(o[:, 0])
        assert hit[key:, 3].all() and not hit[: key // 128 * 128].any()
        hit[:, 3] = False
        assert not hit.any()


@pytest.mark.parametrize("kind", ["usual", "signed"])
def test_position_track(kind):
    """A permuted pack: distances come from the position track."""
    samples = [[wl.Span("causal", 90), wl.Span("group", 130), wl.Span("causal", 41),
                wl.Span("group", 200), wl.Span("causal", 51)],
               [wl.Span("causal", 100), wl.Span("full", 156)], [wl.Span("noise", 128),
                                                                wl.Span("causal", 128)]]
    tr = wl.tracks_from_samples(samples)
    n = len(tr["sample"])
    perm = M.layout_vision_groups(tr["sample"], tr["seg"])
    moved = {x: np.asarray(tr[x])[perm] for x in tr}
    moved["pos"] = perm.astype(np.int32)
    q, k, v, do = _qkvdo(n, 4, 4, 64, 8)
    slopes = _slopes(4, kind)
    s, g, z = device_tracks(moved)
    pos = torch.as_tensor(moved["pos"]).cuda()
    for P, fused in ((1, True), (2, False)):
        pl = M.Plan(s, g, z, INF, P, "ptrr_block", pos=pos)
        for cap in (0.0, 2.0):
            _check(_run(pl, q, k, v, do, M.Score(cap, slopes), fused=fused), q, k, v, do,
                   mask.dense_mask(moved, INF), cap, slopes, moved["pos"])


@pytest.mark.parametrize("cap", [1e-30, 1e-3, 0.1, 1e4, 1e30])
def test_extreme_caps(cap):
    """Caps far below and far above the scores: all weights alike, and no cap at all."""
    n = 512
    tr = wl.random_pack(np.random.default_rng(3), n, max_samples=2)
    q, k, v, do = _qkvdo(n, 2, 2, 64, 3)
    pl = M.Plan(*device_tracks(tr), INF, 1)
    m = mask.dense_mask(tr, INF)
    for fused in (False, True):
        _check(_run(pl, q, k, v, do, M.Score(cap), fused=fused), q, k, v, do, m, cap, None)
    # scores of zero, whatever the cap
    got = _run(pl, torch.zeros_like(q), k, v, do, M.Score(cap))
    _check(got, torch.zeros_like(q), k, v, do, m, cap, None)


@pytest.mark.parametrize("cap", [2.5e3, 4e4, 1e6])
def test_large_products_under_large_caps(cap):
    """Products of some thousands, caps around and above them.  Few keys have weight, and a score
    of size S is off by 2^-22 S (the sum of d products, the polynomial), so the keys and scale are
    chosen for scores up to 0.9 caps or 4000 that differ between keys by less than 1."""
    n, d = 256, 64
    tr = wl.tracks_from_samples([[wl.Span("causal", 200), wl.Span("full", 56)]])
    q, k, v, do = _qkvdo(n, 1, 1, d, 4)
    q.zero_()
    q[..., 0] = 8.0   # exact products: 8 * 8 * 64, and small ones beside them
    q[..., 1] = torch.linspace(-1, 1, n, device="cuda").bfloat16()[:, None]
    k.zero_()
    k[..., 0] = 8.0
    k[..., 1] = torch.linspace(1, -1, n, device="cuda").bfloat16()[:, None]
    scale = min(0.9 * cap, 4000.0) / 64
    q[..., 1] /= scale
    pl = M.Plan(*device_tracks(tr), INF, 1)
    st, o, lse = M.State(n, 1, d), torch.empty_like(q), torch.empty((1, n), device="cuda")
    score = M.Score(cap)
    M.forward(pl, q, k, v, st, o, lse, fused=True, scale=scale, score=score)
    m = mask.dense_mask(tr, INF)
    ref = scored.attention(q, k, v, m, cap, scale=scale, do=do, h=HALF)
    S = scale * 64 + 1
    off = 2.0 ** -21 * S  # the score and its maximum
    # the LSE is a score plus a logarithm, rounded to fp32
    assert (np.abs(_np(lse) - ref["LSE"]) <= off + 2.0 ** -22 * S).all()
    lim = (1 + HALF) * ((1 + 2 * off / HALF) * ref["bound"]["O"] + HALF * np.abs(ref["O"]))
    assert (np.abs(_np(o) - ref["O"]) <= lim + 1e-30).all()
    delta = torch.empty_like(lse)
    dq, dk, dv = (torch.zeros(x.shape, device="cuda") for x in (q, k, v))
    M.backward(pl, q, k, v, o, do, lse, delta, dq, dk, dv, fused=True, scale=scale, score=score)
    pl.check()
    for name, x in zip(("dq", "dk", "dv"), (dq, dk, dv)):
        err = np.abs(_np(x) - ref[name])
        # 1 - tanh^2 is off by 2^-21 of one, 2^-18 of itself at 0.9 caps
        lim = (1 + HALF) * (1 + (8 * off + 2.0 ** -18) / HALF) * ref["bound"][name]
        assert (err <= lim + 1e-6 * scale).all(), (name, (err - lim).max())


@pytest.mark.parametrize("cap", [3.0, 50.0, 55.0, 60.0])
@pytest.mark.parametrize("size", [1e-4, 1.0, 1e6])
def test_saturated_scores(cap, size):
    """Rows whose scores all are near -cap, rows near +cap and rows with both, small and large
    values: caps on both sides of where the forward does without a running maximum (cap log2 e
    of 80)."""
    n, d = 512, 64
    tr = wl.tracks_from_samples([[wl.Span("causal", 300), wl.Span("full", 212)]])
    q, k, v, do = _qkvdo(n, 2, 1, d, 9)
    # scores of 4 caps in size: channel 0 of the keys has signs by thirds
    k[..., 0] = 8.0
    k[150:300, :, 0] = -8.0
    q[..., 0] = 4 * cap / 8 * (-1) ** (torch.arange(n, device="cuda") // 7)[:, None]
    v *= size
    pl = M.Plan(*device_tracks(tr), INF, 2)
    m = mask.dense_mask(tr, INF)
    st, o, lse = M.State(n, 2, d), torch.empty_like(q), torch.empty((2, n), device="cuda")
    ref = scored.attention(q, k, v, m, cap, scale=1.0, do=do, h=HALF)
    for fused in (False, True):
        M.forward(pl, q, k, v, st, o, lse, fused=fused, scale=1.0, score=M.Score(cap))
        pl.check()
        # a score of up to 80 log2 e is off by its roundings, 2^-20 of the cap in all
        off = 2.0 ** -20 * cap
        assert (np.abs(_np(lse) - ref["LSE"]) <= off + 2.0 ** -18).all()
        lim = (1 + HALF) * ((1 + 2 * off / HALF) * ref["bound"]["O"] + HALF * np.abs(ref["O"]))
        assert (np.abs(_np(o) - ref["O"]) <= lim + 1e-30).all()


@pytest.mark.parametrize("kind", ["usual", "steep", "signed"])
@pytest.mark.parametrize("W", [INF, 40])
def test_bias_beside_a_cap_that_bounds_the_scores(kind, W):
    """Heads whose slopes lower scores do without a running maximum, the others in the same launch
    do not; steep slopes leave a row little more than its own key."""
    n, cap = 1024, 50.0
    tr = wl.random_pack(np.random.default_rng(31), n, max_samples=4)
    q, k, v, do = _qkvdo(n, 4, 2, 128, 31, scale=20.0)
    slopes = _slopes(4, kind)
    pl = M.Plan(*device_tracks(tr), W, 2, "ptrr_block")
    m = mask.dense_mask(tr, W)
    assert (m.diagonal() == m.any(1)).all()
    for kw in ({}, {"fused": True}, {"merge": "fp32"}):
        _check(_run(pl, q, k, v, do, M.Score(cap, slopes), **kw), q, k, v, do, m, cap, slopes)


def test_both_ways_to_tanh_in_one_pack():
    """Rows with small and rows with large scores, tile by tile, around the border of 0.75."""
    n = 1024
    tr = wl.tracks_from_samples([[wl.Span("causal", 600), wl.Span("full", 424)]])
    q, k, v, do = _qkvdo(n, 2, 1, 128, 6)
    gain = torch.ones(n, device="cuda")
    gain[::3], gain[1::64], gain[512:] = 0.05, 4.0, 0.3
    q = (q.float() * gain[:, None, None]).bfloat16()
    pl = M.Plan(*device_tracks(tr), INF, 2)
    m = mask.dense_mask(tr, INF)
    for cap in (2.0, 4.0, 8.0):
        _check(_run(pl, q, k, v, do, M.Score(cap), fused=True), q, k, v, do, m, cap, None)


def test_scale_and_merges():
    n = 1024
    tr = wl.config_tracks(2, n)
    q, k, v, do = _qkvdo(n, 2, 2, 64, 7)
    slopes = _slopes(2, "usual")
    pl = M.Plan(*device_tracks(tr), INF, 4, "ptrr_block")
    m = mask.dense_mask(tr, INF)
    for merge, steps in (("fp32", 1), ("bf16", 9)):  # four partials and four merges rounded
        got = _run(pl, q, k, v, do, M.Score(3.0, slopes), merge=merge)
        ref = scored.attention(q, k, v, m, 3.0, _np(slopes), h=HALF)
        # a partial is a mean over its keys: rounding it costs half a step of P |V| at the most
        lim = (1 + HALF) * ((1 + SOFT / HALF + (steps - 1)) * ref["bound"]["O"] +
                            HALF * np.abs(ref["O"]) + 1e-30)
        assert (np.abs(_np(got[0]) - ref["O"]) <= lim).all()
        assert (np.abs(_np(got[1]) - ref["LSE"]) <= SOFT).all()
    st, o, lse = M.State(n, 2, 64), torch.empty_like(q), torch.empty((2, n), device="cuda")
    M.forward(pl, *(pl.permute(x) for x in (q, k, v)), st, o, lse, scale=0.3, fused=True,
              score=M.Score(3.0, slopes))
    ref = scored.attention(q, k, v, m, 3.0, _np(slopes), scale=0.3, h=HALF)
    lim = (1 + HALF) * ((1 + SOFT / HALF) * ref["bound"]["O"] + HALF * np.abs(ref["O"]) + 1e-30)
    assert (np.abs(_np(pl.permute(o, inverse=True)) - ref["O"]) <= lim).all()


def test_no_change_is_the_plain_call():
    """A score without cap and slopes has the plain call's bits; so has a step of the list."""
    n = 1024
    tr = wl.config_tracks(2, n)
    q, k, v, do = _qkvdo(n, 4, 2, 64, 9)
    pl = M.Plan(*device_tracks(tr), INF, 2)
    for kw in ({}, {"needed": True}, {"fused": True}):
        for x, y in zip(_run(pl, q, k, v, do, None, **kw), _run(pl, q, k, v, do, M.Score(), **kw)):
            assert torch.equal(x, y)
    score = M.Score(4.0, _slopes(4, "usual"))
    a, b = M.State(n, 4, 64), M.State(n, 4, 64)
    M.attn_steps(pl, q, k, v, M.ring_schedule(2), a, score=score)
    for r, j, first in M.ring_schedule(2):
        M.attn_step(pl, q, k, v, r, j, b, first=first, score=score)
    o, lse = torch.empty_like(q), torch.empty((4, n), device="cuda")
    M.attn_finalize(pl, a, o, lse)
    for x, y in ((a.o_acc, b.o_acc), (a.m, b.m), (a.l, b.l)):
        assert torch.equal(x, y)
    delta = torch.empty_like(lse)
    M.attn_bwd_prep(pl, o, do, delta)
    g, w = ([torch.zeros(x.shape, device="cuda") for x in (q, k, v)] for _ in range(2))
    for r, j, _ in M.ring_schedule(2):
        M.attn_bwd(pl, q, k, v, do, lse, delta, r, j, *g, score=score)
    M.attn_bwd_steps(pl, q, k, v, do, lse, delta, M.ring_schedule(2), *w, score=score)
    for x, y in zip(g, w):  # the list may take whole rows: summation order
        assert rel_fro(_np(x), _np(y)) <= 1e-4


def test_repeats_streams_and_side_streams():
    n = 2048
    tr = wl.config_tracks(2, n)
    q, k, v, do = _qkvdo(n, 4, 2, 128, 10)
    pl = M.Plan(*device_tracks(tr), INF, 4, "ptrr_block")
    score = M.Score(6.0, _slopes(4, "usual"))
    for fused in (False, True):
        want = _run(pl, q, k, v, do, score, fused=fused)
        again = [_run(pl, q, k, v, do, score, fused=fused),
                 _run(pl, q, k, v, do, score, fused=fused, stream=torch.cuda.Stream())]
        try:
            M.set_side_streams(0)
            again.append(_run(pl, q, k, v, do, score, fused=fused))
        finally:
            M.set_side_streams(4)
        for got in again:
            for x, y in zip(want, got):
                assert torch.equal(x, y)


@pytest.mark.parametrize("hq,hkv,P", [(8, 2, 1), (6, 1, 4), (12, 3, 2)])
def test_grouped_heads_of_small_packs(hq, hkv, P):
    """Few units and grouped heads: the fused backward gives every q head units of its own.  Its
    gradients are within the bounds, add to what the accumulators hold, and repeat."""
    n = 1024
    tr = wl.config_tracks(2, n)
    q, k, v, do = _qkvdo(n, hq, hkv, 64, 13)
    slopes = _slopes(hq, "usual")
    pl = M.Plan(*device_tracks(tr), INF, P)
    score = M.Score(8.0, slopes)
    m = mask.dense_mask(tr, INF)
    got = _run(pl, q, k, v, do, score, fused=True)
    _check(got, q, k, v, do, m, 8.0, slopes)
    for x, y in zip(got, _run(pl, q, k, v, do, score, fused=True)):
        assert torch.equal(x, y)
    lse, delta = got[1].contiguous(), torch.empty_like(got[1])
    M.attn_bwd_prep(pl, got[0], do, delta)
    ones = [torch.ones(x.shape, device="cuda") for x in (q, k, v)]
    M.attn_bwd_fused(pl, q, k, v, do, lse, delta, *ones, score=score)
    for x, y in zip(ones, got[2:]):
        # 1 + g is rounded to fp32 once for every addition to the accumulator (at most the heads
        # of a group, or P steps of a row), to half a step of values below 64
        assert (x - 1 - y).abs().max() <= max(hq // hkv, P) * 64 * 2.0 ** -24 + 1e-6


def test_full_size_rows():
    """The 64K packed configuration: rows of whole short samples against the oracle."""
    cfg = wl.CONFIGS[2]
    tr = wl.config_tracks(2)
    q, k, v, do = _qkvdo(cfg.n, 4, 4, cfg.d, 11)
    slopes = _slopes(4, "usual")
    pl = M.Plan(*device_tracks(tr), INF, cfg.shards, cfg.order)
    got = _run(pl, q, k, v, do, M.Score(20.0, slopes), fused=True)
    st, en = mask.sample_runs(tr)
    starts = np.unique(st)
    lengths = en[starts] - starts
    picks = [starts[i] for i in np.argsort(lengths)[[0, len(lengths) // 4, len(lengths) // 2]]]
    picks.append([s for s in starts if en[s] - s < 2048][-1])
    for a in picks:
        b = int(en[a])
        sub = {x: np.asarray(tr[x])[a:b] for x in ("sample", "seg", "noise")}
        cut = [x[a:b] for x in (q, k, v, do)]
        part = (got[0][a:b], got[1][:, a:b]) + tuple(x[a:b] for x in got[2:])
        _check(part, *cut, mask.dense_mask(sub, INF), 20.0, slopes)


def test_refusals():
    n = 256
    zero = torch.zeros(n, dtype=torch.int32, device="cuda")
    none = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    pl = M.Plan(zero, none, none, INF, 1)
    q, k, v, _ = _qkvdo(n, 2, 2, 64, 1)
    st = M.State(n, 2, 64)
    for cap in (-1.0, float("nan"), float("inf"), 1e31, 1e-31):
        with pytest.raises(M.MarbleError, match="cap"):
            M.attn_fwd_fused(pl, q, k, v, st, score=M.Score(cap))
    with pytest.raises(ValueError):
        M.Score(slopes=torch.zeros(2, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        M.Score(slopes=torch.zeros(2))
    with pytest.raises(ValueError):
        M.Score(slopes=torch.zeros((2, 1), device="cuda"))
    with pytest.raises(ValueError):
        M.attn_fwd_fused(pl, q, k, v, st, score=M.Score(slopes=torch.zeros(3, device="cuda")))
    with pytest.raises(M.MarbleError, match="aligned"):
        M.attn_fwd_fused(pl, q, k, v, st,
                         score=M.Score(slopes=torch.zeros(3, device="cuda")[1:]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(M.MarbleError, match="captured"):
            M.attn_fwd_fused(pl, q, k, v, st, score=M.Score(2.0))
        st.m.zero_()
    M.attn_fwd_fused(pl, q, k, v, st, score=M.Score(2.0))
    pl.check()


@pytest.mark.parametrize("stream", [False, True])
def test_a_layer_with_rotary_positions(stream):
    """What a layer does with the two together: the fused projection's q, k and v normed, rotated
    by (t, h, w) and moved into plan order, attention with capped scores and a bias, its backward,
    and the projection's gradient back in original order."""
    from oracle import rope as R
    n, hq, hkv, d = 1024, 6, 2, 64
    tr = wl.config_tracks(2, n)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    qkv = torch.randn((n, hq + 2 * hkv, d), generator=g, device="cuda").bfloat16()
    do = torch.randn((n, hq, d), generator=g, device="cuda").bfloat16()
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    pos = torch.randint(0, 64, (3, n), generator=g, device="cuda", dtype=torch.int32)
    freq, axis = M.rope_frequencies((16, 8, 8))
    rope = M.Rope(freq, axis)
    slopes = _slopes(hq, "usual")
    pl = M.Plan(*device_tracks(tr), INF, 2, "ptrr_block")
    q, k, v = qkv.split((hq, hkv, hkv), 1)
    score = M.Score(10.0, slopes)
    s = torch.cuda.Stream() if stream else None
    if s:
        s.wait_stream(torch.cuda.current_stream())
    kw = dict(plan=pl, q_weight=wq, k_weight=wk, stream=s)
    qp, kp, vp = M.rope(rope, pos, q, k, v, **kw)
    with torch.cuda.stream(s):
        st = M.State(n, hq, d)
        o, lse = torch.empty_like(qp), torch.empty((hq, n), device="cuda")
        delta = torch.empty_like(lse)
        dq, dk, dv = (torch.zeros(x.shape, device="cuda") for x in (qp, kp, vp))
        dp = pl.permute(do, stream=s)
        out = torch.empty_like(qkv)
    M.forward(pl, qp, kp, vp, st, o, lse, fused=True, score=score, stream=s)
    M.backward(pl, qp, kp, vp, o, dp, lse, delta, dq, dk, dv, fused=True, score=score, stream=s)
    dwq, dwk = M.rope_bwd(rope, pos, dq, dk, dv, q=q, k=k, out=out.split((hq, hkv, hkv), 1), **kw)[3:]
    pl.check(stream=s)
    torch.cuda.synchronize()
    # the attention of the rotated q and k that the kernel rounded (their own error is tested with
    # the rotary calls), in original order
    qr, kr, vr = (pl.permute(x, inverse=True) for x in (qp, kp, vp))
    ref = scored.attention(qr, kr, vr, mask.dense_mask(tr, INF), 10.0, _np(slopes), None, None, do,
                           HALF)
    p = pos.cpu().numpy()
    for got, x, w, name, dw in ((out[:, :hq], q, wq, "dq", dwq),
                                (out[:, hq:hq + hkv], k, wk, "dk", dwk)):
        x, w = _np(x), _np(w)
        want, want_w = R.backward(ref[name], x, p, freq, axis, "halves", w)
        # turning keeps the size of an error, the norm's gradient multiplies it by r max |w| at
        # most; the result is rounded once
        r = 1 / np.sqrt((x * x).mean(-1) + 1e-6)
        noise = np.sqrt(ref["noise"][name].sum())
        err = np.linalg.norm(_np(got) - want)
        assert err <= r.max() * np.abs(w).max() * noise + HALF * np.linalg.norm(want)
        # a weight's gradient is the sum over the rows of gradient times x r, at most sqrt(d)
        assert np.linalg.norm(_np(dw) - want_w) <= np.sqrt(d) * np.sqrt(x.shape[0] * x.shape[1]) * \
            noise
    err = np.linalg.norm(_np(out[:, hq + hkv:]) - ref["dv"])
    assert err <= np.sqrt(ref["noise"]["dv"].sum()) + HALF * np.linalg.norm(ref["dv"])
