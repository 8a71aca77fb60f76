"""The paged cache on the GPU: what is written, quantised and read back, against the fp64 oracle.
Codes, scales and bf16 values are compared for equality: every rounding in them is one rounding
of an exact number."""
import math

import numpy as np
import pytest
import torch

import context_attention_metadata_gb300 as M
from cached_testlib import DTYPES, E4M3, Batch, bf16, codes_of, np64, quantised
from oracle import cached as C

pytestmark = pytest.mark.gpu
KINDS = sorted(DTYPES)


def _rows(n, hkv, d, seed, fused=True):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kv = bf16(gen, (n, 2 * hkv, d), 1.5)
    k, v = kv.split(hkv, 1)
    return (k, v) if fused else (k.contiguous(), v.contiguous())


def _expect(batch, k, v, before, order=None):
    """The pool after writing rows k, v (host float64) over `before` = (codes, scales)."""
    codes, scales = before[0].copy(), None if before[1] is None else before[1].copy()
    x = np.stack([np64(k), np64(v)], 1)
    for row, b, p, g, t in C.places(batch.table, batch.lens, batch.start, batch.page, len(x)):
        at = row if order is None else order[row]
        if scales is None:
            codes[g, :, :, t] = x[at]
        else:
            codes[g, :, :, t], scales[g, :, :, t] = quantised(x[at], batch.kind)
    return codes, scales


def _equal(got, want):
    np.testing.assert_array_equal(got[0], want[0])
    if want[1] is not None:
        np.testing.assert_array_equal(got[1], want[1])


CASES = [  # lens, counts (None: one row each), hkv, d, page
    ([1], None, 1, 64, 16),
    ([17, 0, 64, 33], None, 8, 128, 32),
    ([5, 300, 77], [5, 41, 77], 3, 64, 48),
    ([1000, 3, 129, 64], [999, 3, 0, 64], 2, 128, 64),
    ([2, 50], [5, 50], 5, 128, 256),        # three rows before position 0
    ([4100], [4100], 8, 64, 128),
    (list(range(70)), None, 2, 64, 16),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,counts,hkv,d,page", CASES)
@pytest.mark.parametrize("fused", [True, False])
def test_write(kind, lens, counts, hkv, d, page, fused):
    batch = Batch(kind, lens, counts, hkv, d, page, seed=len(lens), stride_pad=16)
    k, v = _rows(batch.n + 3, hkv, d, 1, fused)  # rows behind the last sequence are not written
    if counts is None:
        k, v = k[:batch.n], v[:batch.n]
    before = batch.values()
    whole = batch.pool.view(torch.int8).clone()
    M.cache_write(batch.cache, batch.seqs, k, v)
    got, want = batch.values(), _expect(batch, k, v, before)
    _equal(got, want)
    batch.seqs.check()
    # bytes between the pages
    assert torch.equal(batch.pool.view(torch.int8)[:, -16:], whole[:, -16:])


@pytest.mark.parametrize("kind", KINDS)
def test_write_one_of_both(kind):
    batch = Batch(kind, [40, 9], None, 2, 64, 16)
    k, v = _rows(2, 2, 64, 3)
    before = batch.values()
    M.cache_write(batch.cache, batch.seqs, None, v)
    want = _expect(batch, k, v, before)
    want[0][:, 0] = before[0][:, 0]
    if want[1] is not None:
        want[1][:, 0] = before[1][:, 0]
    _equal(batch.values(), want)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_heads_of_every_size(kind):
    """Tops over all of bf16's exponents and mantissas, the channels up to the top itself and
    multiples that land on ties."""
    rng = np.random.default_rng(5)
    low = 1 if kind == "int8" else 16  # (e4m3's scale stops at 2^-126)
    tops = np.arange(low << 7, 255 << 7, 13, dtype=np.int64)
    d, n = 64, len(tops)
    bits = rng.integers(0, tops[:, None] + 1, (n, d))
    near = np.maximum(tops[:, None] - rng.integers(0, 1 << 10, (n, d)), 0)
    bits = np.where(rng.random((n, d)) < 0.7, near, bits)
    bits[:, 7] = tops
    bits |= rng.integers(0, 2, (n, d)) << 15
    x = torch.as_tensor(bits.astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    x[::9, 10:20] = (x[::9, 7:8].double() / 254 * torch.arange(1, 21, 2)).bfloat16()
    x = x[:, None].cuda()
    batch = Batch(kind, [n], [n], 1, d, 64)
    M.cache_write(batch.cache, batch.seqs, x, x)
    got = batch.values()
    ref = np64(x)[:, 0]
    codes, scales = quantised(ref, kind)
    for row, b, p, g, t in C.places(batch.table, batch.lens, batch.start, 64, n):
        np.testing.assert_array_equal(got[0][g, 0, 0, t], codes[row])
        assert got[1][g, 0, 0, t] == scales[row]
    for row in range(0, n, 97):  # and by rationals
        c, s = C.quantise_head(ref[row], kind)
        np.testing.assert_array_equal(c, codes[row])
        assert s == scales[row]


@pytest.mark.parametrize("kind", KINDS)
def test_special_heads(kind):
    batch = Batch(kind, [6], [6], 2, 128, 16, fill=False)
    k, v = _rows(6, 2, 128, 4, fused=False)
    k[0, 0] = 0
    k[1, 1, 5] = math.inf
    k[2, 0, 127] = math.nan
    v[3, 1, 0] = -math.inf
    v[4] = 0
    M.cache_write(batch.cache, batch.seqs, k, v)
    rk, rv = M.cache_read(batch.cache, batch.seqs, n=6)
    for x, r in ((k, rk), (v, rv)):
        x, r = np64(x), np64(r)
        if kind == "bf16":
            np.testing.assert_array_equal(r, x)
            continue
        bad = ~np.isfinite(x).all(-1)
        assert np.isnan(r[bad]).all() and np.isfinite(r[~bad]).all()
        assert (r[(x == 0).all(-1)] == 0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,counts,hkv,d,page", CASES)
def test_read(kind, lens, counts, hkv, d, page):
    batch = Batch(kind, lens, counts, hkv, d, page, seed=7)
    n = batch.n + (5 if counts is not None else 0)
    out = torch.full((n, 2 * hkv, d), 3.0, dtype=torch.bfloat16, device="cuda")
    M.cache_read(batch.cache, batch.seqs, out=out.split(hkv, 1))
    want = np.full((n, 2, hkv, d), 3.0)
    want[:batch.n] = 0  # rows before position 0
    for row, b, p, g, t in C.places(batch.table, batch.lens, batch.start, page, n):
        want[row, 0], want[row, 1] = batch.k[b][p], batch.v[b][p]
    # code * scale in fp32 (int8: rounded there first), then bf16
    want = torch.as_tensor(want).float().bfloat16().double().numpy()
    got = np64(out).reshape(n, 2, hkv, d)
    if kind == "int8":
        off = np.abs(got - want)  # two roundings of one product may part at a tie
        assert (off <= np.abs(want) * 2.0 ** -7).all() and (off > 0).mean() < 1e-4
    else:
        np.testing.assert_array_equal(got, want)
    batch.seqs.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shards,order", [(1, "contiguous"), (4, "ptrr_block")])
def test_plan_order(kind, shards, order):
    """Rows in plan order: written by their original places, read into plan order."""
    n, hkv, d = 1024, 2, 64
    counts = [500, 1, 300, 211]  # twelve rows of padding behind them
    lens = [500, 40, 310, 211]
    z = torch.zeros(n, dtype=torch.int32, device="cuda")
    none = torch.full_like(z, -1)
    plan = M.Plan(z, none, none, M.WINDOW_INF, shards, order)
    batch = Batch(kind, lens, counts, hkv, d, 32)
    k, v = _rows(n, hkv, d, 9)
    kp, vp = plan.permute(k.contiguous()), plan.permute(v.contiguous())
    before = batch.values()
    M.cache_write(batch.cache, batch.seqs, kp, vp, plan=plan)
    _equal(batch.values(), _expect(batch, k, v, before))
    rk, rv = M.cache_read(batch.cache, batch.seqs, plan=plan)
    ok, ov = M.cache_read(batch.cache, batch.seqs, n=n)
    assert torch.equal(rk, plan.permute(ok)) and torch.equal(rv, plan.permute(ov))
    assert not ok[1012:].any() and ok[:1012].any(-1).all()
    with pytest.raises(M.MarbleError, match="n_tokens"):
        M.cache_write(batch.cache, batch.seqs, kp[:512], vp[:512], plan=plan)
    plan.close()
    with pytest.raises(ValueError, match="closed"):
        M.cache_write(batch.cache, batch.seqs, kp, vp, plan=plan)


def test_offsets_beyond_32_bits():
    pages, hkv, page, d = 21000, 8, 64, 128  # 5.5 GB with keys and values side by side
    pool = torch.empty((pages, 2, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    cache = M.Cache(pool[:, 0], pool[:, 1])
    table = torch.tensor([[pages - 1, 3], [pages - 2, pages - 3]], dtype=torch.int32).cuda()
    lens = torch.tensor([64, 128], dtype=torch.int32).cuda()
    start = torch.tensor([0, 64, 192], dtype=torch.int32).cuda()
    k, v = _rows(192, hkv, d, 2)
    seqs = M.Sequences(table, lens, start)
    M.cache_write(cache, seqs, k, v)
    rk, rv = M.cache_read(cache, seqs, n=192)
    assert torch.equal(rk, k) and torch.equal(rv, v)
    assert torch.equal(pool[pages - 2, 1].transpose(0, 1), v[64:128])


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_bad_metadata_touches_nothing(kind):
    """Pages and lengths out of bounds: the other sequences are right, the pool elsewhere keeps
    its bytes, the status says so."""
    batch = Batch(kind, [40, 20, 33, 10], [40, 20, 33, 10], 2, 64, 16)
    batch.seqs.table[1, 1] = 1 << 30
    batch.seqs.table[2, 0] = -5
    batch.seqs.lens[3] = 1 << 20
    k, v = _rows(103, 2, 64, 5)
    before = batch.values()
    good = Batch.__new__(Batch)
    good.__dict__.update(batch.__dict__)
    want = [before[0].copy(), None if before[1] is None else before[1].copy()]
    x = np.stack([np64(k), np64(v)], 1)
    for row, b, p, g, t in C.places(batch.table, batch.lens, batch.start, 16, 103):
        if b == 3 or (b == 1 and p >= 16) or (b == 2 and p < 16):
            continue
        if kind == "bf16":
            want[0][g, :, :, t] = x[row]
        else:
            want[0][g, :, :, t], want[1][g, :, :, t] = quantised(x[row], kind)
    M.cache_write(batch.cache, batch.seqs, k, v)
    _equal(batch.values(), want)
    with pytest.raises(M.MarbleError, match="out of bounds"):
        batch.seqs.check()
    batch.status.zero_()
    M.cache_read(batch.cache, batch.seqs, n=103)
    assert int(batch.status) == M.SEQS_BAD
    # a start that decreases, and one that passes the rows
    batch = Batch(kind, [16, 16, 16], [4, 4, 4], 2, 64, 16)
    batch.seqs.start.copy_(torch.tensor([0, 8, 4, 1 << 20], dtype=torch.int32))
    M.cache_write(batch.cache, batch.seqs, k[:12], v[:12])
    assert int(batch.status) == M.SEQS_BAD


@pytest.mark.parametrize("kind", KINDS)
def test_another_stream_and_a_graph(kind):
    """A captured step is replayed with other rows and lengths, on another stream than the one
    the tensors were made on."""
    batch = Batch(kind, [33, 7, 64], None, 4, 128, 16)
    k, v = _rows(3, 4, 128, 11, fused=False)
    out = torch.zeros((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        M.cache_write(batch.cache, batch.seqs, k, v)
        M.cache_read(batch.cache, batch.seqs, out=out.split(4, 1))
    for step in range(3):
        k2, v2 = _rows(3, 4, 128, 20 + step, fused=False)
        lens = [33 + step, 7 + step, 64 - step]
        batch.lens = np.array(lens)
        batch.seqs.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        k.copy_(k2)
        v.copy_(v2)
        before = batch.values()
        graph.replay()
        _equal(batch.values(), _expect(batch, k2, v2, before))
        a, b = M.cache_read(batch.cache, batch.seqs)
        assert torch.equal(torch.cat((a, b), 1), out)
    with torch.cuda.stream(side):
        M.cache_write(batch.cache, batch.seqs, k, v, stream=side)
        a, b = M.cache_read(batch.cache, batch.seqs, stream=side)
    side.synchronize()
    assert torch.equal(torch.cat((a, b), 1), out)


def test_refusals():
    batch = Batch("int8", [40, 9], None, 2, 64, 16)
    k, v = _rows(2, 2, 64, 3)
    c, s = batch.cache, batch.seqs
    for bad in ((k.float(), v), (k[:1], v), (k[:, :1], v[:, :1]), (k[..., :32], v[..., :32]),
                (k.cpu(), v), (k.transpose(0, 1), v), (None, None)):
        with pytest.raises(ValueError):
            M.cache_write(c, s, *bad)
    with pytest.raises(M.MarbleError, match="one row a sequence"):
        M.cache_write(c, s, k[:1], v[:1])
    with pytest.raises(M.MarbleError, match="stride"):
        odd = torch.empty((2, 2 * 64 + 4), dtype=torch.bfloat16, device="cuda")
        M.cache_write(c, s, odd[:, :128].view(2, 2, 64), None)
    bcache = Batch("bf16", [40, 9], None, 2, 64, 16)
    inside = bcache.body[0, 0].transpose(0, 1)[:2].contiguous()
    view = bcache.pool.view(-1)[:2 * 128].view(2, 2, 64)
    with pytest.raises(M.MarbleError, match="overlap the cache"):
        M.cache_read(bcache.cache, bcache.seqs, out=(view, None))
    with pytest.raises(M.MarbleError, match="overlap"):
        M.cache_read(bcache.cache, bcache.seqs, out=(inside, inside))
    with pytest.raises(M.MarbleError, match="overlap each other"):
        bad = M.Cache(bcache.body[:, 0], bcache.body[:, 0])
        M.cache_write(bad, bcache.seqs, k, v)
    with pytest.raises(ValueError):
        M.Cache(c.k, c.v)  # no scales
    with pytest.raises(ValueError):
        M.Cache(c.k, c.v, c.k_scale[:, :1], c.v_scale)
    with pytest.raises(ValueError):
        M.Cache(c.k.transpose(1, 2), c.v.transpose(1, 2), c.k_scale, c.v_scale)
    with pytest.raises(M.MarbleError, match="page_tokens"):
        M.cache_write(M.Cache.empty(4, 2, 24, 64), s, k, v)
    with pytest.raises(M.MarbleError, match="head dim"):
        x = torch.zeros((2, 2, 32), dtype=torch.bfloat16, device="cuda")
        M.cache_write(M.Cache.empty(4, 2, 16, 32), s, x, x)
    with pytest.raises(ValueError):
        M.Sequences(s.table.long(), s.lens)
    with pytest.raises(ValueError):
        M.Sequences(s.table, s.lens[:1])
    with pytest.raises(ValueError):
        M.Sequences(s.table, s.lens, s.lens)
    with pytest.raises(ValueError, match="n, the number"):
        start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        M.cache_read(c, M.Sequences(s.table, s.lens, start))
    assert int(batch.status) == 0


def test_copies_have_their_own_tensors():
    import copy
    a = M.Cache.empty(4, 2, 16, 64, torch.float8_e4m3fn)
    b = copy.deepcopy(a)
    assert b._c.k == b.k.data_ptr() != a.k.data_ptr()
    assert b._c.v_scale == b.v_scale.data_ptr() != a.v_scale.data_ptr()
    with pytest.raises(AttributeError):
        a.k = b.k


def test_empty_calls():
    batch = Batch("bf16", [5], [5], 2, 64, 16)
    before = batch.values()
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    M.cache_write(batch.cache, batch.seqs, none, none)
    _equal(batch.values(), before)
    no = M.Sequences(batch.seqs.table[:0], batch.seqs.lens[:0])
    M.cache_write(batch.cache, no, none, none)
    assert M.cache_read(batch.cache, no)[0].shape == (0, 2, 64)
