"""Attention over the paged cache on the GPU against the fp64 oracle; the tolerances are derived
in cached_testlib.attn_bounds."""
import numpy as np
import pytest
import torch

import context_attention_metadata_gb300 as M
from cached_testlib import DTYPES, Batch, bf16, check_attn, np64, quantised
from oracle import cached as C

pytestmark = pytest.mark.gpu
KINDS = sorted(DTYPES)


def _q(n, hq, d, seed, size=2.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 50)
    return (torch.randn((n, hq, d), generator=gen, device="cuda") * size).bfloat16()


def _slopes(hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device="cuda")


def _run(batch, q, window=None, span=False, cap=0.0, slopes=None, scale=None, **kw):
    score = M.Score(cap, slopes) if cap or slopes is not None else None
    return M.attn_cached(batch.cache, batch.seqs, q, scale=scale or 0.0,
                         window=M.WINDOW_INF if window is None else window, span=span, score=score,
                         **kw)


CASES = [  # lens, counts, hkv, group, d, page
    ([1], None, 1, 1, 64, 16),
    ([64], None, 2, 1, 128, 64),
    ([65, 31, 32, 33], None, 2, 4, 128, 16),
    ([0, 5, 0, 127, 128, 129], None, 1, 7, 64, 32),      # idle places
    ([2000], None, 2, 8, 128, 64),                       # one item over many CTAs
    ([700, 3, 1500], [1, 3, 5], 3, 2, 64, 48),           # pages that end inside a chunk
    ([300, 17, 64], [4, 0, 7], 1, 8, 128, 256),          # 32 and 56 rows; a sequence without any
    ([90, 40], [20, 40], 2, 4, 64, 16),                  # more than 64 rows: several tiles
    ([10, 200], [16, 2], 1, 16, 128, 32),                # rows before position 0
    (list(range(1, 61)), None, 2, 2, 64, 16),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,counts,hkv,group,d,page", CASES)
def test_plain(kind, lens, counts, hkv, group, d, page):
    batch = Batch(kind, lens, counts, hkv, d, page, seed=len(lens))
    q = _q(batch.n, hkv * group, d, 1)
    o, lse = _run(batch, q)
    check_attn(batch, q, o, lse)
    batch.seqs.check()
    again = _run(batch, q)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,span,cap,bias,scale", [
    (1, False, 0.0, False, None), (33, False, 0.0, False, None), (0, False, 0.0, False, None),
    (7, True, 0.0, False, None), (0, True, 0.0, False, None), (None, True, 0.0, True, None),
    (None, False, 20.0, False, None), (100, False, 0.0, True, 0.3), (64, True, 5.0, True, None),
    (None, False, 1e-30, False, None), (None, False, 1e30, False, None)])
def test_masks_and_scores(kind, window, span, cap, bias, scale):
    for lens, counts, d, page in (([700, 3, 130, 0], [4, 3, 6, 1], 128, 64),
                                  ([257, 64], [9, 1], 64, 16)):
        batch = Batch(kind, lens, counts, 2, d, page, seed=3)
        q = _q(batch.n, 6, d, 2)
        slopes = _slopes(6) if bias else None
        o, lse = _run(batch, q, window, span, cap, slopes, scale)
        check_attn(batch, q, o, lse, window, span, cap, slopes, scale)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group,hint", [(1, 1), (1, 20), (3, 8), (5, 8), (16, 1), (32, 1), (80, 1)])
def test_tiles_of_rows(kind, group, hint):
    """Every tile height, and more rows than the hint says."""
    batch = Batch(kind, [333, 20], [3, 20], 2, 64, 32, seed=group)
    q = _q(batch.n, 2 * group, 64, 3)
    o, lse = _run(batch, q, new_tokens=hint)
    check_attn(batch, q, o, lse)


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(kind):
    """More sequences than a CTA has threads, most of them idle or short."""
    rng = np.random.default_rng(1)
    lens = np.where(rng.random(700) < 0.5, 0, rng.integers(0, 90, 700))
    lens[[13, 699]] = 1500
    batch = Batch(kind, lens, None, 1, 64, 16)
    q = _q(700, 2, 64, 4)
    o, lse = _run(batch, q)
    check_attn(batch, q, o, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,group,counts,lens", [
    (128, 2, None, [30000, 5, 21003]), (64, 4, None, [30000, 5, 21003]),
    (128, 4, [7, 1, 16], [30000, 5, 21003]),
    # items of up to and of more than 16 rows in turn: the places of the ring change hands
    (128, 4, [1, 8, 3, 5, 4, 6, 2, 8] * 3, [700, 2900, 33, 1500, 64, 900, 2000, 1200] * 3),
    (64, 8, [4, 1, 3, 2] * 6, [500, 77, 1900, 640] * 6)])
def test_the_ring_goes_round(kind, d, group, counts, lens):
    """Enough keys that every CTA fills its ring many times over."""
    batch = Batch(kind, lens, counts, 6, d, 64, seed=5)
    q = _q(batch.n, 6 * group, d, 10)
    o, lse = _run(batch, q)
    check_attn(batch, q, o, lse)
    batch.seqs.check()
    for _ in range(20):
        again = _run(batch, q)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("kind", KINDS)
def test_strided_rows_and_outputs(kind):
    """q as a slice of a projection, o as a slice, no lse, rows behind the last sequence."""
    batch = Batch(kind, [100, 61], [2, 3], 2, 128, 16)
    qkv = _q(8, 10, 128, 5)
    q = qkv[:, 1:7]
    wide = torch.full((8, 9, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((6, 8), 5.0, device="cuda")
    _run(batch, q, out=(wide[:, 2:8], lse))
    check_attn(batch, q[:5], wide[:5, 2:8], lse[:, :5])
    assert (wide[5:] == 7).all() and (wide[:, :2] == 7).all() and (wide[:, 8:] == 7).all()
    assert (lse[:, 5:] == 5).all()
    other = torch.empty_like(wide)
    _run(batch, q, out=(other[:, 2:8], None))
    assert torch.equal(other[:5, 2:8], wide[:5, 2:8])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_large_and_small_values(kind):
    """Scores far from each other and scales of very different sizes: the weights' units follow
    the largest scale, which comes late."""
    batch = Batch(kind, [400], None, 1, 128, 16)
    if kind == "e4m3":
        f = torch.ones(400)
        f[100] = 2.0 ** 12
        f[399] = 2.0 ** 14
        page, slot = np.arange(400) // 16, np.arange(400) % 16
        g = torch.as_tensor(batch.table[0][page].astype(np.int64)).cuda()
        batch.scale[g, 1, 0, torch.as_tensor(slot).cuda()] *= f.cuda()
        batch.v[0] = batch.v[0] * f.double().numpy()[:, None, None]
    for size in (1e-3, 30.0):
        q = _q(1, 4, 128, 6, size)
        o, lse = _run(batch, q)
        check_attn(batch, q, o, lse)


@pytest.mark.parametrize("kind", KINDS)
def test_only_needed_pages_are_looked_at(kind):
    """Entries in front of a window and behind a sequence may hold anything."""
    batch = Batch(kind, [500, 130], None, 2, 64, 16)
    q = _q(2, 4, 64, 7)
    want = _run(batch, q, 100)
    table = batch.seqs.table
    table[0, :25] = 1 << 30       # 400 = 499 - 99: positions 400 .. 499 are seen
    table[1, :1] = -1
    table[1, 9:] = 1 << 29
    o, lse = _run(batch, q, 100)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    batch.seqs.check()


@pytest.mark.parametrize("kind", KINDS)
def test_bad_metadata(kind):
    batch = Batch(kind, [500, 130, 64], None, 2, 64, 16)
    q = _q(3, 4, 64, 8)
    want = _run(batch, q)
    batch.seqs.table[0, 3] = 1 << 30
    o, lse = _run(batch, q)
    assert torch.equal(o[1:], want[0][1:]) and torch.equal(lse[:, 1:], want[1][:, 1:])
    with pytest.raises(M.MarbleError, match="out of bounds"):
        batch.seqs.check()
    batch.status.zero_()
    batch.seqs.lens[1] = 1 << 24
    batch.seqs.lens[2] = -3
    batch.seqs.table.clamp_(0, 0)
    _run(batch, q)
    assert int(batch.status) == M.SEQS_BAD


@pytest.mark.parametrize("kind", KINDS)
def test_shared_prefix_and_one_page_twice(kind):
    """Pages in two tables, and the same page at two places of one."""
    batch = Batch(kind, [64, 64], None, 2, 64, 16)
    table = batch.seqs.table
    table[1, :3] = table[0, :3]
    table[1, 3] = table[0, 1]
    batch.k[1] = np.concatenate([batch.k[0][:48], batch.k[0][16:32]])
    batch.v[1] = np.concatenate([batch.v[0][:48], batch.v[0][16:32]])
    q = _q(2, 4, 64, 9)
    o, lse = _run(batch, q)
    check_attn(batch, q, o, lse)


@pytest.mark.parametrize("kind", KINDS)
def test_streams_and_graphs(kind):
    """Two graphs with a workspace each, replayed on two streams at once with other lengths; an
    eager call beside them."""
    batches = [Batch(kind, [3000, 40], None, 2, 128, 64, seed=s) for s in (1, 2)]
    qs = [_q(2, 8, 128, s) for s in (1, 2)]
    outs = [(torch.empty_like(q), torch.empty((8, 2), device="cuda")) for q in qs]
    wss = [torch.empty(M.ATTN_CACHED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
           for _ in qs]
    graphs, sides = [], [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for batch, q, out, ws, side in zip(batches, qs, outs, wss, sides):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            _run(batch, q, out=out, workspace=ws)
    for lens in ([3000, 40], [1777, 33], [1, 2]):
        for b in batches:
            b.lens = np.array(lens)
            b.seqs.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        kept = [(b.k, b.v) for b in batches]
        torch.cuda.synchronize()
        for _ in range(20):
            for g, side in zip(graphs, sides):
                with torch.cuda.stream(side):
                    g.replay()
        eager = _run(batches[0], qs[0])
        torch.cuda.synchronize()
        for b, q, (o, lse), side in zip(batches, qs, outs, sides):
            b.k, b.v = [x[:n] for x, n in zip(b.k, lens)], [x[:n] for x, n in zip(b.v, lens)]
            check_attn(b, q, o, lse)
        assert torch.equal(eager[0], outs[0][0]) and torch.equal(eager[1], outs[0][1])
        for b, (k, v) in zip(batches, kept):
            b.k, b.v = k, v
    side = sides[0]
    for b in batches:
        b.seqs.lens.copy_(torch.tensor([3000, 40], dtype=torch.int32))
        b.lens = np.array([3000, 40])
    side.wait_stream(torch.cuda.current_stream())
    o, lse = _run(batches[1], qs[1], stream=side)
    side.synchronize()
    check_attn(batches[1], qs[1], o, lse)


def test_positions_up_to_the_last():
    """A table that names one page 32,767 times: as many positions as there may be.  Every key counts
    32,767 times, so o is the page's own and lse ln 32,767 more.  Sums of fp32 lose up to 2^-24 a
    term: a thread adds 2^31 / (2 CTAs x 148 SMs x 4 warps x 8 lanes) weights, 1.4%, and the
    matrix unit as many products of 16 keys, twice that; both enter o."""
    page = 65536
    batch = Batch("int8", [page], None, 1, 64, page, spare=0)
    q = _q(1, 4, 64, 12)
    o1, l1 = _run(batch, q)
    check_attn(batch, q, o1, l1)
    reps = (2 ** 31 - 65536) // page
    assert reps == 32767
    table = torch.zeros((1, reps), dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seqs = M.Sequences(table, torch.tensor([reps * page], dtype=torch.int32).cuda(), None, status)
    o, lse = M.attn_cached(batch.cache, seqs, q)
    seqs.check()
    size = np64(o1).__abs__() + np.abs(batch.v[0]).max() * 0.043
    assert (np.abs(np64(o) - np64(o1)) <= 0.043 * size + 2 * 2.0 ** -8 * size).all()
    assert (np.abs(np64(lse) - np64(l1) - np.log(reps)) < 0.015).all()
    # the end of it alone, in a window
    ow, lw = M.attn_cached(batch.cache, seqs, q, window=page)
    torch.testing.assert_close(ow, o1, rtol=2 ** -6, atol=2 ** -8)
    torch.testing.assert_close(lw, l1, rtol=0, atol=1e-4)
    seqs.lens.add_(1)  # one more is refused by the kernel
    M.attn_cached(batch.cache, seqs, q)
    assert int(status) == M.SEQS_BAD


@pytest.mark.parametrize("kind", KINDS)
def test_one_table_on_two_streams_and_threads(kind):
    """Calls on the same sequences at the same time, from two threads on two streams, have
    workspaces of their own."""
    import threading
    batch = Batch(kind, [9000, 77], None, 2, 64, 64)
    qs = [_q(2, 8, 64, s) for s in (20, 21)]
    want = [_run(batch, q) for q in qs]
    torch.cuda.synchronize()
    bad = []

    def work(q, w):
        stream = torch.cuda.Stream()
        for _ in range(50):
            o, lse = _run(batch, q, stream=stream)
            stream.synchronize()
            if not (torch.equal(o, w[0]) and torch.equal(lse, w[1])):
                bad.append(1)

    threads = [threading.Thread(target=work, args=a) for a in zip(qs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("kind", KINDS)
def test_prompt_then_tokens(kind):
    """The calls as they are used: a packed prompt through rope, the cache and the packed
    attention, then tokens one by one (and three at once) through rope, the cache and the cached
    attention, against attention over everything that was cached."""
    n, hq, hkv, d = 512, 4, 2, 128
    counts = np.array([200, 17, 290])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    sample = torch.as_tensor(np.repeat([0, 1, 2, 3], [*counts, n - counts.sum()])).int().cuda()
    none = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    plan = M.Plan(sample, none, none, M.WINDOW_INF, 4, "ptrr_block")
    rope = M.Rope(*M.rope_frequencies((64,)))
    at = torch.as_tensor(np.concatenate([np.arange(c) for c in (*counts, n - counts.sum())]))
    qkv = bf16(gen, (n, hq + 2 * hkv, d))
    q, k, v = M.rope(rope, at.int().cuda()[None], *qkv.split((hq, hkv, hkv), 1), plan=plan)
    batch = Batch(kind, counts + 16, counts, hkv, d, 16, fill=False)  # room for 16 tokens more
    batch.seqs.lens.copy_(torch.as_tensor(counts).int())
    M.cache_write(batch.cache, batch.seqs, k, v, plan=plan)
    back = plan.permute(k, inverse=True), plan.permute(v, inverse=True)

    def cached(x):
        x = np64(x)
        if kind == "bf16":
            return x
        c, s = quantised(x, kind)
        return c * s[..., None]

    ends = np.cumsum(counts)
    batch.k = [cached(back[0][e - c:e]) for e, c in zip(ends, counts)]
    batch.v = [cached(back[1][e - c:e]) for e, c in zip(ends, counts)]
    # the prompt's own attention, against the cached form of its last row
    state = M.State(n, hq, d)
    o = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((hq, n), device="cuda")
    M.forward(plan, q, k, v, state, o, lse)
    last = torch.as_tensor(ends - 1).cuda()
    one = M.Sequences(batch.seqs.table, batch.seqs.lens)
    oc, lc = M.attn_cached(batch.cache, one, plan.permute(q, inverse=True)[last])
    if kind == "bf16":
        packed = plan.permute(o, inverse=True)[last].float()
        rel = (packed - oc.float()).norm() / packed.norm()
        assert rel < 0.01  # both round to bf16, the packed one its weights too
        perm = plan.export("perm").long()
        assert torch.allclose(lse[:, torch.argsort(perm)][:, last], lc, atol=1e-3)
    lens = counts.copy()
    for step, new in enumerate((1, 1, 3, 1)):
        lens = lens + new
        batch.lens = lens
        batch.start = np.arange(4) * new
        batch.seqs.lens.add_(new)
        seqs = one if new == 1 else M.Sequences(batch.seqs.table, batch.seqs.lens,
                                                torch.as_tensor(batch.start).int().cuda())
        pos = (batch.seqs.lens[:, None] - new + torch.arange(new, device="cuda")).reshape(1, -1)
        qkv = bf16(gen, (3 * new, hq + 2 * hkv, d))
        q1, k1, v1 = M.rope(rope, pos.int().contiguous(), *qkv.split((hq, hkv, hkv), 1))
        M.cache_write(batch.cache, seqs, k1, v1)
        o1, l1 = M.attn_cached(batch.cache, seqs, q1)
        for b in range(3):
            batch.k[b] = np.concatenate([batch.k[b], cached(k1[b * new:(b + 1) * new])])
            batch.v[b] = np.concatenate([batch.v[b], cached(v1[b * new:(b + 1) * new])])
        check_attn(batch, q1, o1, l1)
    # a chunk behind its prefix: the whole sequences into a pack's keys and values
    rk, rv = M.cache_read(batch.cache, M.Sequences(
        batch.seqs.table, batch.seqs.lens,
        torch.as_tensor(np.concatenate([[0], np.cumsum(lens)])).int().cuda()), n=int(lens.sum()))
    want = np.concatenate(batch.k)
    half = 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8)
    assert (np.abs(np64(rk) - want) <= half).all()
    batch.seqs.check()


def test_refusals():
    batch = Batch("bf16", [40, 9], None, 2, 64, 16)
    q = _q(2, 4, 64, 1)
    c, s = batch.cache, batch.seqs
    for bad in (q.float(), q[..., :32], q.cpu(), q[0], q.transpose(0, 1)):
        with pytest.raises(ValueError):
            M.attn_cached(c, s, bad)
    with pytest.raises(M.MarbleError, match="one row a sequence"):
        M.attn_cached(c, s, q[:1])
    with pytest.raises(M.MarbleError, match="multiple of hkv"):
        M.attn_cached(c, s, q[:, :3])
    with pytest.raises(M.MarbleError, match="window"):
        M.attn_cached(c, s, q, window=-1)
    with pytest.raises(M.MarbleError, match="scale"):
        M.attn_cached(c, s, q, scale=float("nan"))
    with pytest.raises(M.MarbleError, match="cap"):
        M.attn_cached(c, s, q, score=M.Score(-1.0))
    with pytest.raises(ValueError, match="slopes"):
        M.attn_cached(c, s, q, score=M.Score(0.0, _slopes(3)))
    with pytest.raises(M.MarbleError, match="overlaps"):
        M.attn_cached(c, s, q, out=(q, None))
    with pytest.raises(ValueError, match="workspace"):
        M.attn_cached(c, s, q, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        M.attn_cached(c, s, q, out=(torch.empty_like(q), torch.empty((2, 4), device="cuda")))
    with pytest.raises(ValueError):
        M.attn_cached(c, s, q, out=(q.float(), None))
    o, lse = M.attn_cached(c, M.Sequences(s.table[:0], s.lens[:0]), q[:0])
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
