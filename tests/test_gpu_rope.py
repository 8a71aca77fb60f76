"""Rotary positions on the GPU against the fp64 oracle.

Tolerances.  A result is rounded to bf16 once: half a step, 2^-8 of its value.  Before that it
is fp32: with u = 2^-24, the angle is off by 1.6 u (half a step of a fraction of a half turn,
times pi), sine and cosine by 2 u, the products and their sum by 2 u, a norm by 16 u (the sum of
squares 8, the root and the quotient 4, the products 4), together under 24 u of the pair's size."""
import ctypes

import numpy as np
import pytest
import torch

import context_attention_metadata_gb300 as M
import workloads as wl
from oracle import rope as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = torch.finfo(torch.bfloat16).eps / 2


def _tensors(n, hq, hkv, d, seed, fused=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qkv = torch.randn((n, hq + 2 * hkv, d), generator=g, device="cuda").bfloat16()
    parts = qkv.split((hq, hkv, hkv), 1)
    return parts if fused else tuple(x.contiguous() for x in parts)


def _grads(n, hq, hkv, d, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 77)
    return tuple(torch.randn((n, h, d), generator=g, device="cuda") for h in (hq, hkv, hkv))


def _weights(d, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 5)
    return tuple(1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2))


def _positions(axes, n, seed, top=100000):
    rng = np.random.default_rng(seed)
    return torch.as_tensor(rng.integers(-top, top, (axes, n)).astype(np.int32)).cuda()


def _sections(rot, axes):
    p = rot // 2
    return [p - (axes - 1) * (p // axes)] + [p // axes] * (axes - 1)


def _np(t):
    return t.detach().double().cpu().numpy()


def _pair_size(x, rot, pairing):
    """The size of the pair that each channel belongs to."""
    a, b = R.pair_channels(rot, pairing)
    s = np.abs(x)
    s[..., a] = s[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return s


def _check_forward(y, x, rope, pos, w, eps):
    x, p = _np(x), pos.cpu().numpy()
    w = None if w is None else _np(w)
    ref = R.forward(x, p, rope.inv_freq, rope.axis, rope.pairing, w, eps)
    size = _pair_size(R.normed(x, w, eps), rope.rot_dim, rope.pairing)
    err = np.abs(_np(y) - ref)
    assert (err <= HALF * np.abs(ref) + 24 * U * (1 + HALF) * size).all(), \
        (err - HALF * np.abs(ref)).max()


CASES = [  # n, hq, hkv, d, rot, axes, layout, pairing, norm
    (1, 1, 1, 64, 16, 1, "sections", "halves", False),
    (1, 32, 8, 128, 128, 3, "sections", "halves", True),
    (2, 3, 1, 64, 64, 2, "axial", "adjacent", True),
    (7, 14, 2, 64, 32, 1, "sections", "adjacent", False),
    (61, 5, 5, 128, 112, 4, "interleaved", "halves", True),
    (129, 9, 3, 128, 48, 3, "axial", "adjacent", True),
    (1000, 2, 2, 64, 48, 3, "interleaved", "halves", True),
    (4099, 7, 1, 128, 128, 2, "axial", "halves", False),
    (5003, 12, 3, 64, 64, 3, "sections", "adjacent", False),
]


@pytest.mark.parametrize("n,hq,hkv,d,rot,axes,layout,pairing,norm", CASES)
@pytest.mark.parametrize("fused", [True, False])
def test_forward(n, hq, hkv, d, rot, axes, layout, pairing, norm, fused):
    q, k, v = _tensors(n, hq, hkv, d, n, fused)
    pos = _positions(axes, n, n)
    rope = M.Rope(*M.rope_frequencies(_sections(rot, axes), 10000.0, layout), pairing)
    wq, wk = _weights(d, n) if norm else (None, None)
    qo, ko, vo = M.rope(rope, pos, q, k, v, q_weight=wq, k_weight=wk, eps=1e-5)
    assert qo.is_contiguous() and ko.is_contiguous()
    _check_forward(qo, q, rope, pos, wq, 1e-5)
    _check_forward(ko, k, rope, pos, wk, 1e-5)
    assert torch.equal(vo, v)


@pytest.mark.parametrize("n,hq,hkv,d,rot,axes,layout,pairing,norm", CASES)
def test_gradient(n, hq, hkv, d, rot, axes, layout, pairing, norm):
    q, k, _ = _tensors(n, hq, hkv, d, n)
    dq, dk, dv = _grads(n, hq, hkv, d, n)
    pos = _positions(axes, n, n)
    rope = M.Rope(*M.rope_frequencies(_sections(rot, axes), 10000.0, layout), pairing)
    w = _weights(d, n) if norm else (None, None)
    gq, gk, gv, dwq, dwk = M.rope_bwd(rope, pos, dq, dk, dv, q=q, k=k, q_weight=w[0],
                                      k_weight=w[1], eps=1e-5)
    assert torch.equal(gv, dv.bfloat16())
    p = pos.cpu().numpy()
    for got, dw, g, x, wt in ((gq, dwq, dq, q, w[0]), (gk, dwk, dk, k, w[1])):
        x, g, wt = _np(x), _np(g), None if wt is None else _np(wt)
        ref, rw = R.backward(g, x, p, rope.inv_freq, rope.axis, pairing, wt, 1e-5)
        size = _pair_size(g, rot, pairing)
        if wt is not None:
            # the terms of dx: r g w and x r mean(g w x r), each of whose factors is off by
            # the bound above, the mean of d products by as much again
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
            gw = size * np.abs(wt)
            size = 3 * (r * gw + np.abs(x) * r * r * (gw * np.abs(x) * r).mean(-1, keepdims=True))
        err = np.abs(_np(got) - ref)
        assert (err <= HALF * np.abs(ref) + 24 * U * (1 + HALF) * size).all()
        if wt is None:
            assert dw is None
            continue
        # each product is off by 48 u; a thread adds up to 100 rows one after another, and the
        # lanes', warps', CTAs' sums 50 more
        bound = 200 * U * (_pair_size(g, rot, pairing) * np.abs(x) * r).sum((0, 1))
        assert (np.abs(_np(dw) - rw) <= bound).all()


def test_gradient_against_differences():
    """The kernel's gradient against differences of the fp64 definition along random directions."""
    n, hq, hkv, d = 33, 4, 2, 64
    q, k, _ = _tensors(n, hq, hkv, d, 3)
    dq, dk, _ = _grads(n, hq, hkv, d, 3)
    pos = _positions(2, n, 3)
    rope = M.Rope(*M.rope_frequencies((20, 12)), "halves")
    wq, wk = _weights(d, 3)
    gq, gk, _, dwq, dwk = M.rope_bwd(rope, pos, dq, dk, q=q, k=k, q_weight=wq, k_weight=wk)
    rng = np.random.default_rng(0)
    p, h = pos.cpu().numpy(), 1e-5
    for x, g, w, got, dw in ((q, dq, wq, gq, dwq), (k, dk, wk, gk, dwk)):
        x, g, w = _np(x), _np(g), _np(w)

        def loss(x_, w_):
            return (g * R.forward(x_, p, rope.inv_freq, rope.axis, "halves", w_, 1e-6)).sum()

        for _ in range(4):
            e, ew = rng.standard_normal(x.shape), rng.standard_normal(d)
            diff = (loss(x + h * e, w) - loss(x - h * e, w)) / (2 * h)
            # bf16's rounding of every entry, and 1e-6 of the terms for the rest
            assert abs(diff - (_np(got) * e).sum()) <= \
                (HALF * np.abs(_np(got) * e)).sum() + 1e-6 * np.abs(_np(got) * e).sum()
            diff = (loss(x, w + h * ew) - loss(x, w - h * ew)) / (2 * h)
            assert abs(diff - (_np(dw) * ew).sum()) <= 1e-4 * np.abs(_np(dw) * ew).sum()


@pytest.mark.parametrize("order,P", [("contiguous", 1), ("ptrr_block", 4)])
@pytest.mark.parametrize("norm", [False, True])
def test_plan_order(order, P, norm):
    """With a plan: the same bits as without one, moved as marble_permute moves them; and the
    gradient undoes the move."""
    n, hq, hkv, d = 2048, 6, 2, 64
    tr = wl.config_tracks(1)
    s, g, z = (torch.as_tensor(np.asarray(tr[x], np.int32)).cuda()
               for x in ("sample", "seg", "noise"))
    pl = M.Plan(s, g, z, wl.WINDOW_INF, P, order)
    q, k, v = _tensors(n, hq, hkv, d, 4)
    pos = _positions(3, n, 4)
    rope = M.Rope(*M.rope_frequencies((16, 8, 8)))
    wq, wk = _weights(d, 4) if norm else (None, None)
    kw = dict(q_weight=wq, k_weight=wk)
    here = M.rope(rope, pos, q, k, v, **kw)
    there = M.rope(rope, pos, q, k, v, plan=pl, **kw)
    for a, b in zip(here, there):
        assert torch.equal(pl.permute(a), b)
    grads = _grads(n, hq, hkv, d, 4)
    a = M.rope_bwd(rope, pos, *grads, q=q, k=k, **kw)
    moved = [pl.permute(x) for x in grads]
    fused = torch.empty((n, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    b = M.rope_bwd(rope, pos, *moved, plan=pl, q=q, k=k, out=fused.split((hq, hkv, hkv), 1), **kw)
    for x, y in zip(a[:3], b[:3]):
        assert torch.equal(x, y)
    if norm:
        for x, y in zip(a[3:], b[3:]):  # the rows are summed in another order: 200 u each
            assert (x - y).abs().max() <= 400 * U * n * hq
    with pytest.raises(ValueError):
        M.rope(rope, pos[:, :1024].contiguous(), q[:1024], k[:1024], v[:1024], plan=pl)


def test_far_positions():
    """The last positions of 32 bits are as exact as the first, in both signs."""
    far = [0, 1, -1, 2**24 + 1, 2**31 - 1, -2**31, 2**31 - 129, 123456789]
    n = len(far)
    q, k, _ = _tensors(n, 4, 2, 128, 9)
    pos = torch.tensor([far], dtype=torch.int32, device="cuda")
    for freq in (M.rope_frequencies((64,))[0], -M.rope_frequencies((64,), 7.0)[0],
                 np.linspace(-9, 9, 64)):
        rope = M.Rope(freq)
        qo, ko, _ = M.rope(rope, pos, q, k)
        # freq itself has 53 bits, and 2^31 times its last one is 2^-22 of a radian: the bound
        # gets the oracle's share of that, 2^31 * 2^-53 * |freq|
        slack = 2.0 ** -22 * np.abs(freq).max()
        for y, x in ((qo, q), (ko, k)):
            ref = R.forward(_np(x), pos.cpu().numpy(), rope.inv_freq, rope.axis, "halves")
            size = _pair_size(_np(x), 128, "halves")
            assert (np.abs(_np(y) - ref) <= HALF * np.abs(ref) + (24 * U + slack) * size).all()


def test_infinities_stay_in_their_pairs():
    """Without a norm a channel's infinity or NaN reaches its pair alone, and channels that are
    not rotated are copied."""
    for pairing in ("halves", "adjacent"):
        q, _, _ = _tensors(5, 2, 1, 64, 1, fused=False)
        q[1, 0, 3], q[2, 1, 50], q[3, 0, 60] = float("inf"), float("nan"), float("-inf")
        rope = M.Rope(M.rope_frequencies((16,))[0], pairing=pairing)
        pos = _positions(1, 5, 1)
        y = M.rope(rope, pos, q)[0]
        assert torch.equal(y[..., 32:].view(torch.int16), q[..., 32:].view(torch.int16))
        a, b = R.pair_channels(32, pairing)
        mate = int(b[list(a).index(3)]) if 3 in a else int(a[list(b).index(3)])
        bad = ~torch.isfinite(y[..., :32])
        bad[1, 0, 3] = bad[1, 0, mate] = False
        assert not bad.any()


def test_single_token_and_batch_agree():
    """A token's result has the same bits alone, in a batch, in place and in a long sequence."""
    n, hq, hkv, d = 3000, 8, 2, 128
    q, k, v = _tensors(n, hq, hkv, d, 6)
    pos = _positions(3, n, 6)
    rope = M.Rope(*M.rope_frequencies((32, 16, 16)))
    wq, wk = _weights(d, 6)
    kw = dict(q_weight=wq, k_weight=wk)
    full = M.rope(rope, pos, q, k, v, **kw)
    for a, b in ((0, 1), (17, 18), (100, 164), (2999, 3000)):
        part = M.rope(rope, pos[:, a:b].contiguous(), q[a:b], k[a:b], v[a:b], **kw)
        for x, y in zip(full, part):
            assert torch.equal(x[a:b], y)
    own = [x.clone() for x in (q, k, v)]
    got = M.rope(rope, pos, *own, out=own, **kw)
    for x, y, z in zip(full, own, got):
        assert torch.equal(x, y) and y.data_ptr() == z.data_ptr()
    only_q = M.rope(rope, pos, q, q_weight=wq)
    assert torch.equal(only_q[0], full[0]) and only_q[1] is None


def test_gradient_of_some_tensors_and_in_place():
    n, hq, hkv, d = 200, 4, 2, 64
    q, k, _ = _tensors(n, hq, hkv, d, 8, fused=False)
    dq, dk, dv = _grads(n, hq, hkv, d, 8)
    pos = _positions(1, n, 8)
    rope = M.Rope(M.rope_frequencies((32,))[0], pairing="adjacent")
    wq, wk = _weights(d, 8)
    full = M.rope_bwd(rope, pos, dq, dk, dv, q=q, k=k, q_weight=wq, k_weight=wk)
    one = M.rope_bwd(rope, pos, dq, q=q, q_weight=wq)
    assert torch.equal(one[0], full[0]) and one[4] is None
    only_k = M.rope_bwd(rope, pos, dq, dk, dv, k=k, k_weight=wk)
    assert torch.equal(only_k[1], full[1]) and only_k[3] is None
    # The rows are spread over the warps by the heads of the call, so that the weights' sums run
    # in another order: each is within 200 u (test_gradient) of the sum of its terms' sizes, the
    # two within 400 u of one another.
    for a, b, g, x in ((one[3], full[3], dq, q), (only_k[4], full[4], dk, k)):
        g, x = _pair_size(_np(g), 64, "adjacent"), np.abs(_np(x))
        terms = (g * x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)).sum((0, 1))
        assert (np.abs(_np(a) - _np(b)) <= 400 * U * terms).all()
    # into the forward's inputs themselves
    q2, k2 = q.clone(), k.clone()
    M.rope_bwd(rope, pos, dq, dk, q=q2, k=k2, q_weight=wq, k_weight=wk, out=(q2, k2, None))
    assert torch.equal(q2, full[0]) and torch.equal(k2, full[1])
    # an empty batch: no gradient, the weights' are zero
    e = M.rope_bwd(rope, pos[:, :0].contiguous(), dq[:0], dk[:0], dv[:0], q=q[:0], k=k[:0],
                   q_weight=wq, k_weight=wk)
    assert e[0].shape == (0, hq, d) and (e[3] == 0).all() and (e[4] == 0).all()
    assert M.rope(rope, pos[:, :0].contiguous(), q[:0], k[:0])[0].shape == (0, hq, d)


def test_large_offsets():
    """More than 2^31 elements: rows at both ends and around the 2^31st element."""
    n, hq, hkv, d = 600_000, 20, 5, 128
    q, k, v = _tensors(n, hq, hkv, d, 2)
    pos = _positions(2, n, 2)
    rope = M.Rope(*M.rope_frequencies((32, 32), 10000.0, "axial"))
    wq, wk = _weights(d, 2)
    qo, ko, vo = M.rope(rope, pos, q, k, v, q_weight=wq, k_weight=wk, eps=1e-5)
    edge = 2**31 // ((hq + 2 * hkv) * d)
    rows = torch.as_tensor([0, 1, edge - 1, edge, edge + 1, n - 2, n - 1]).cuda()
    _check_forward(qo[rows], q[rows], rope, pos[:, rows], wq, 1e-5)
    _check_forward(ko[rows], k[rows], rope, pos[:, rows], wk, 1e-5)
    assert torch.equal(vo, v)
    del qo, ko, vo
    g = [x.float() for x in (q, k)]
    out = M.rope_bwd(rope, pos, *g, q=q, k=k, q_weight=wq, k_weight=wk, eps=1e-5)
    some = M.rope_bwd(rope, pos[:, rows].contiguous(), *(x[rows] for x in g),
                      q=q[rows], k=k[rows], q_weight=wq, k_weight=wk, eps=1e-5)
    for x, y in zip(out[:2], some[:2]):
        assert torch.equal(x[rows], y)


def test_streams_graphs_and_repeats():
    """On another stream, captured and replayed with new inputs, and twice over: the same bits."""
    n, hq, hkv, d = 1500, 6, 3, 64
    q, k, v = _tensors(n, hq, hkv, d, 12, fused=False)
    grads = _grads(n, hq, hkv, d, 12)
    pos = _positions(2, n, 12)
    rope = M.Rope(*M.rope_frequencies((16, 16)))
    wq, wk = _weights(d, 12)
    kw = dict(q_weight=wq, k_weight=wk)

    def both(stream=None):
        return M.rope(rope, pos, q, k, v, stream=stream, **kw) + \
            M.rope_bwd(rope, pos, *grads, q=q, k=k, stream=stream, **kw)

    want = both()
    for x, y in zip(want, both()):
        assert torch.equal(x, y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = both(side)
    side.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for seed in (12, 13):
        q2, k2, v2 = _tensors(n, hq, hkv, d, seed, fused=False)
        for a, b in zip((q, k, v), (q2, k2, v2)):
            a.copy_(b)
        graph.replay()
        for x, y in zip(both(), got):
            assert torch.equal(x, y)


def test_captured_with_a_plan():
    """A captured call leaves the plan usable and destroyable."""
    n = 1024
    zero = torch.zeros(n, dtype=torch.int32, device="cuda")
    none = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    pl = M.Plan(zero, none, none, wl.WINDOW_INF, 2, "ptrr_block")
    q, k, v = _tensors(n, 2, 2, 64, 14)
    pos = _positions(1, n, 14)
    rope = M.Rope(M.rope_frequencies((32,))[0])
    want = M.rope(rope, pos, q, k, v, plan=pl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = M.rope(rope, pos, q, k, v, plan=pl)
    graph.replay()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    pl.check()
    torch.cuda.synchronize()
    assert M.lib().marble_plan_destroy(pl.handle) == M.OK
    pl._h = None


def test_refusals_on_the_gpu():
    n, hq, hkv, d = 64, 4, 2, 64
    q, k, v = _tensors(n, hq, hkv, d, 1, fused=False)
    pos = _positions(2, n, 1)
    rope = M.Rope(*M.rope_frequencies((16, 16)))
    w = _weights(d, 1)[0]
    both = torch.zeros((n + 1, hq, d), dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: M.rope(rope, pos, both[:n], out=(both[1:], None, None)),       # shifted overlap
        lambda: M.rope(rope, pos, q, k, v, out=(q, k, k)),                     # k written twice
        lambda: M.rope(M.Rope(*M.rope_frequencies((16, 8, 8))), pos, q),       # axis 2 of two
        lambda: M.rope_bwd(rope, pos, *_grads(n, hq, hkv, d, 1), q_weight=w),  # q is missing
        lambda: M.rope(rope, pos.float(), q),
        lambda: M.rope(rope, pos[0], q),
        lambda: M.rope(rope, pos, q.float()),
        lambda: M.rope(rope, pos, q.transpose(0, 1)),
        lambda: M.rope(rope, pos, q, k[:5]),
        lambda: M.rope(rope, pos, q, k, v[:, :1]),
        lambda: M.rope(rope, pos, q, q_weight=w.bfloat16()),
        lambda: M.rope(rope, pos, q, q_weight=w[:32]),
        lambda: M.rope(rope, pos, q.cpu()),
        lambda: M.rope(rope, pos, q, out=(k, None, None)),
        lambda: M.rope(rope, pos, q[..., :48].contiguous()),                   # d
    ]
    for f in bad:
        with pytest.raises((ValueError, M.MarbleError)):
            f()
    plan_q = torch.empty((2048, 2, 64), dtype=torch.bfloat16, device="cuda")
    tr = wl.config_tracks(1)
    pl = M.Plan(*(torch.as_tensor(np.asarray(tr[x], np.int32)).cuda()
                  for x in ("sample", "seg", "noise")), wl.WINDOW_INF, 4)
    with pytest.raises(M.MarbleError, match="overlap"):  # no rewriting in place through a plan
        M.rope(rope, _positions(2, 2048, 1), plan_q, plan=pl, out=(plan_q, None, None))
    # a stride that is not a multiple of 16 bytes, and a base that is not aligned
    odd = torch.empty(n * (hq * d + 4), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(M.MarbleError, match="stride"):
        M.rope(rope, pos, odd.as_strided((n, hq, d), (hq * d + 4, d, 1)))
    with pytest.raises(M.MarbleError, match="aligned"):
        M.rope(rope, pos, odd[4:4 + n * hq * d].view(n, hq, d))
    assert ctypes.sizeof(M._Heads) == 64


def test_rows_beyond_any_memory_are_refused():
    """2^30 tokens 2^39 elements apart: more bytes than an address has, refused before any launch."""
    q = torch.empty((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    rope = M.Rope(*M.rope_frequencies((32,)))
    c = rope._c(pos, None, None, 1e-6)
    far = M._Heads(q.data_ptr(), None, None, 1 << 39, 0, 0, 1, 0, 64)
    with pytest.raises(M.MarbleError, match="stride"):
        M._call("marble_rope", None, 1 << 30, ctypes.byref(c), ctypes.byref(far),
                ctypes.byref(far), M._stream(None))
