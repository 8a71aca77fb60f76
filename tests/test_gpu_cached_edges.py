"""Attention over the paged cache at the ends of its number ranges, and what of the cache it must not
depend on.  Tolerances: cached_testlib.attn_bounds, with what a test adds derived beside it."""
import numpy as np
import pytest
import torch

import context_attention_metadata_gb300 as M
from cached_testlib import HALF, Batch, attn_bounds, codes_of, np64
from oracle import cached as C

pytestmark = pytest.mark.gpu


def _q(n, hq, d, seed, size=2.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 90)
    return (torch.randn((n, hq, d), generator=gen, device="cuda") * size).bfloat16()


def _slots(batch, b, pos):
    """(pages, slots) of positions of sequence b, as index tensors."""
    g = torch.as_tensor(batch.table[b][pos // batch.page].astype(np.int64)).cuda()
    return g, torch.as_tensor(pos % batch.page).cuda()


def _set_v_scales(batch, b, pos, change):
    """v's scales of the positions become change(scales), and what the oracle gets follows."""
    g, t = _slots(batch, b, pos)
    s = change(batch.scale[g, 1, :, t])
    batch.scale[g, 1, :, t] = s
    codes = batch.body.view(torch.int8)[g, 1, :, t].view(batch.body.dtype)
    batch.v[b][pos] = codes_of(codes) * np64(s)[..., None]


UNIT = 2.0 ** -120  # the least unit of the weights times v's scale


@pytest.mark.parametrize("kind,least,code", [("e4m3", 2.0 ** -126, 448), ("int8", 0.0, 127)])
@pytest.mark.parametrize("tiny", ["all", "first", "last"])
@pytest.mark.parametrize("counts,group,d,window", [
    (None, 4, 128, None), ([3, 2], 4, 64, 150), ([8, 5], 8, 64, None), ([2, 6], 3, 128, 333)])
def test_values_near_fp32s_lower_end(kind, least, code, tiny, counts, group, d, window):
    """v's scales down to the least that cache_write leaves (2^-126, or denormal), heads of zeros
    among them, alone, in front of ordinary ones and behind them.  The weights' unit is 2^-120 at
    least, so the fp16 step below its normal range is 2^-25 / 64 of that for every key, times its
    code; o's own rounding below bf16's normal range is 2^-134, fp32's below its own 2^-149."""
    lens = [700, 90]
    batch = Batch(kind, lens, counts, 2, d, 16, seed=11)
    for b, length in enumerate(lens):
        edge = length // 2
        pos = {"all": np.arange(length), "first": np.arange(edge),
               "last": np.arange(edge, length)}[tiny]
        _set_v_scales(batch, b, pos, lambda s: (s * 2.0 ** -123).clamp(min=least))
        _set_v_scales(batch, b, pos[1::5], lambda s: s * 0)
    q = _q(batch.n, 2 * group, d, 1)
    o, lse = M.attn_cached(batch.cache, batch.seqs, q,
                           window=M.WINDOW_INF if window is None else window)
    ref = C.attention(np64(q), batch.k, batch.v, batch.lens, batch.start, window)
    vmax = max(np.abs(x).max() for x in batch.v)
    bo, bl = attn_bounds(ref, kind, d, max(lens), vmax)
    bo = bo + (1 + HALF["bf16"]) * max(lens) * 2.0 ** -31 * UNIT * code + 2.0 ** -134 + 2.0 ** -147
    assert (np.abs(np64(o) - ref["o"]) <= bo).all()
    assert (np.abs(np64(lse) - ref["lse"]) <= bl).all()
    batch.seqs.check()


def _fill_unseen(batch, value, lo):
    """Slots that no row sees become `value`: the keys' and values' channels, or their scales over
    codes of a large number.  lo: the first position that some row of each sequence sees."""
    seen = torch.zeros((batch.body.shape[0], batch.page), dtype=torch.bool, device="cuda")
    for b, length in enumerate(batch.lens):
        seen[_slots(batch, b, np.arange(min(lo[b], length), length))] = True
    g, t = (~seen).nonzero(as_tuple=True)
    if batch.kind == "bf16":
        batch.body[g, :, :, t] = value
    else:
        batch.body.view(torch.int8)[g, :, :, t] = 126  # 448 as e4m3
        batch.scale[g, :, :, t] = value


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("cap,bias", [(50.0, False), (50.0, True), (0.0, True), (0.0, False)])
@pytest.mark.parametrize("lens,counts,group,d,page,window", [
    ([5, 700, 33], None, 4, 128, 16, None), ([5, 700, 33], None, 4, 64, 16, None),
    ([70, 300, 2], [3, 4, 2], 4, 128, 16, 40), ([70, 300, 9], [8, 5, 3], 8, 64, 32, 37)])
def test_what_no_row_sees_changes_no_bit(kind, cap, bias, lens, counts, group, d, page, window):
    """Unused slots of the pool and what is left of earlier calls in the kernel's ring may hold any
    finite number too.  Scores are far below the cap, where tanh is taken by its polynomial; those of
    the unseen keys would be beyond its reach."""
    batch = Batch(kind, lens, counts, 2, d, page, seed=21)
    new = np.ones(len(lens), int) if counts is None else np.asarray(counts)
    lo = np.zeros(len(lens), int) if window is None else \
        np.maximum(np.asarray(lens) - new - window + 1, 0)
    q = _q(batch.n, 2 * group, d, 2, 0.5)
    slopes = torch.tensor([2.0 ** -(4 + h) for h in range(2 * group)], device="cuda") if bias \
        else None
    score = M.Score(cap, slopes) if cap or bias else None
    # a batch whose keys are all large, to leave them in the ring
    large = Batch(kind, [4000] * 40, None, 2, d, page, seed=22, fill=False)
    _fill_unseen(large, 3e3, [4000] * 40)
    large_q = _q(40, 2 * group, d, 3)

    def run():
        return M.attn_cached(batch.cache, batch.seqs, q, score=score,
                             window=M.WINDOW_INF if window is None else window)

    want = None
    for value in (0.0, 3e3, -3e3, 0.0):
        _fill_unseen(batch, value, lo)
        for _ in range(3):
            M.attn_cached(large.cache, large.seqs, large_q, score=score)
            got = run()
            want = want or got
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(bool(torch.isfinite(x).all()) for x in want)


@pytest.mark.parametrize("call", ["write", "read"])
@pytest.mark.parametrize("start,lens", [
    ([0, 10, 5, 20], [16, 16, 16]),      # one that decreases; the rows' own look-ups miss it
    ([0, 8, 20, 20], [16, 16, -3]),      # lens of sequences without rows
    ([0, 20, 20, 20], [32, 1 << 20, 0]),
    ([0, 20, 20, 1 << 20], [32, 0, 0])])
def test_bad_metadata_of_sequences_that_no_row_leads_to(call, start, lens):
    """What is out of bounds is told whichever sequence holds it."""
    batch = Batch("bf16", [32, 32, 32], [8, 8, 4], 2, 64, 16)
    k, v = (_q(20, 2, 64, s) for s in (4, 5))

    def run():
        if call == "write":
            M.cache_write(batch.cache, batch.seqs, k, v)
        else:
            M.cache_read(batch.cache, batch.seqs, n=20)

    run()
    batch.seqs.check()
    batch.seqs.start.copy_(torch.tensor(start, dtype=torch.int32))
    batch.seqs.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    run()
    assert int(batch.status) == M.SEQS_BAD


def test_many_sequences_without_rows_are_all_looked_at():
    batch = Batch("bf16", [16] * 3000, [1] * 2 + [0] * 2998, 1, 64, 16)
    k, v = (_q(2, 1, 64, s) for s in (4, 5))
    M.cache_write(batch.cache, batch.seqs, k, v)
    batch.seqs.check()
    for b in (2, 224, 225, 1500, 2999):
        batch.seqs.lens[b] = 17
        M.cache_write(batch.cache, batch.seqs, k, v)
        assert int(batch.status) == M.SEQS_BAD
        batch.seqs.lens[b] = 16
        batch.status.zero_()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_windows_beyond_32_bits(kind):
    """A window is any whole number: none of its bits are cut off on the way."""
    batch = Batch(kind, [90, 40], [2, 3], 2, 64, 16)
    q = _q(5, 4, 64, 6)
    want = M.attn_cached(batch.cache, batch.seqs, q)
    for window in (1 << 31, 1 << 32, (1 << 32) + 5, 1 << 70):
        got = M.attn_cached(batch.cache, batch.seqs, q, window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for window in (-1, -(1 << 31) - 1, -(1 << 32), 5 - (1 << 32)):
        with pytest.raises(M.MarbleError, match="window"):
            M.attn_cached(batch.cache, batch.seqs, q, window=window)
    # the hint too
    got = M.attn_cached(batch.cache, batch.seqs, q, new_tokens=(1 << 32) + 1)
    ref = C.attention(np64(q), batch.k, batch.v, batch.lens, batch.start)
    assert torch.isfinite(got[1]).all()
    bo, bl = attn_bounds(ref, kind, 64, 90, max(np.abs(x).max() for x in batch.v))
    assert (np.abs(np64(got[0]) - ref["o"]) <= bo).all()
    assert (np.abs(np64(got[1]) - ref["lse"]) <= bl).all()
    many = M.attn_cached(batch.cache, batch.seqs, q, new_tokens=1 << 20)
    assert torch.equal(got[0], many[0]) and torch.equal(got[1], many[1])


@pytest.mark.parametrize("handed", [True, False])
def test_check_waits_for_the_calls_stream(handed):
    """The status of calls on another stream than the current one."""
    batch = Batch("bf16", [40, 9], None, 2, 64, 16)
    q = _q(2, 4, 64, 7)
    M.attn_cached(batch.cache, batch.seqs, q)
    batch.seqs.check()
    batch.seqs.table[0, 1] = 1 << 30
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    M.attn_cached(batch.cache, batch.seqs, q, stream=side)
    with pytest.raises(M.MarbleError, match="out of bounds"):
        if handed:
            batch.seqs.check(stream=side)
        else:
            with torch.cuda.stream(side):
                batch.seqs.check()
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind,counts,group,d", [
    ("bf16", None, 4, 128), ("int8", [8] * 12, 8, 128), ("e4m3", [1, 4] * 6, 8, 64)])
def test_waits_that_run_out_of_time(kind, counts, group, d):
    """With a limit of a nanosecond some wait of a long batch gives up: the call ends, the status says
    so, and after the limit is put back the same call is right."""
    lens = [20000 + 777 * b for b in range(12)]
    batch = Batch(kind, lens, counts, 2, d, 16, fill=False)
    batch.body.view(torch.int16 if kind == "bf16" else torch.int8).zero_()
    if batch.scale is not None:
        batch.scale.zero_()
    q = _q(batch.n, 2 * group, d, 8)
    run = lambda: M.attn_cached(batch.cache, batch.seqs, q)
    M.set_wait_limit_ns(1)
    try:
        for _ in range(20):
            run()
        torch.cuda.synchronize()
    finally:
        M.set_wait_limit_ns(2_000_000_000)
    assert int(batch.status) == M.SEQS_TIMEOUT
    with pytest.raises(M.MarbleError, match="wait") as e:
        batch.seqs.check()
    assert e.value.status == M.ERR_TIMEOUT
    batch.status.zero_()
    o, lse = run()
    batch.seqs.check()
    # All scores are 0, all values are 0: weights and their sums are whole numbers below 2^24, so
    # lse has log2's error (2^-23 of it), that of ln 2 and the product's (2^-24 each).
    new = np.ones(12, int) if counts is None else np.asarray(counts)
    seen = np.concatenate([n - c + 1 + np.arange(c) for n, c in zip(lens, new)])
    assert not o.any()
    np.testing.assert_allclose(np64(lse), np.broadcast_to(np.log(seen), lse.shape),
                               rtol=2.0 ** -22)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("cap", [1e-30, 1e-3, 1.0, 8.0, 50.0, 1e4, 1e30])
@pytest.mark.parametrize("size", [1e-3, 1.0, 20.0])
def test_caps_of_every_size(kind, cap, size):
    """What a cap may add to a score's error is 4 u of the score: the polynomial and tanhf are off
    relative to it (2^-22.7 and 2 ulp), and the cap's own roundings are counted with the factors."""
    for counts, group, d, page in (([2, 3], 3, 128, 16), (None, 5, 64, 64)):
        batch = Batch(kind, [600, 45], counts, 2, d, page, seed=31)
        q = _q(batch.n, 2 * group, d, 9, size)
        o, lse = M.attn_cached(batch.cache, batch.seqs, q, score=M.Score(cap, None))
        ref = C.attention(np64(q), batch.k, batch.v, batch.lens, batch.start, cap=cap)
        vmax = max(np.abs(x).max() for x in batch.v)
        bo, bl = attn_bounds(ref, kind, d, 600, vmax)
        more = 4 * 2.0 ** -24 * np.minimum(cap, ref["terms"])
        bl = bl + more
        bo = bo + (1 + HALF["bf16"]) * 2 * more.T[..., None] * ref["abs"]
        assert (np.abs(np64(o) - ref["o"]) <= bo).all()
        assert (np.abs(np64(lse) - ref["lse"]) <= bl).all()
        if cap == 1e30:  # as without one: a score's cube over cap^2 is nothing
            plain = M.attn_cached(batch.cache, batch.seqs, q)
            assert (np.abs(np64(lse) - np64(plain[1])) <= 2 * bl).all()
            assert (np.abs(np64(o) - np64(plain[0])) <= 2 * bo).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("cap", [50.0, 1e30])
@pytest.mark.parametrize("down", [20, 40])
def test_caps_of_small_queries_and_large_keys(kind, cap, down):
    """Scores of ordinary size whose factors are not, far below the cap."""
    batch = Batch(kind, [600, 45], [2, 3], 2, 128, 16, seed=32)
    for b, length in enumerate(batch.lens):
        g, t = _slots(batch, b, np.arange(length))
        batch.scale[g, 0, :, t] *= 2.0 ** down
        batch.k[b] = batch.k[b] * 2.0 ** down
    q = (_q(batch.n, 6, 128, 10).float() * 2.0 ** -down).bfloat16()
    o, lse = M.attn_cached(batch.cache, batch.seqs, q, score=M.Score(cap, None))
    ref = C.attention(np64(q), batch.k, batch.v, batch.lens, batch.start, cap=cap)
    bo, bl = attn_bounds(ref, kind, 128, 600, max(np.abs(x).max() for x in batch.v))
    more = 4 * 2.0 ** -24 * np.minimum(cap, ref["terms"])
    bo = bo + (1 + HALF["bf16"]) * 2 * more.T[..., None] * ref["abs"]
    assert (np.abs(np64(lse) - ref["lse"]) <= bl + more).all()
    assert (np.abs(np64(o) - ref["o"]) <= bo).all()


def test_more_than_2_to_30_sequences():
    """All places of a batch but the last are without rows: the search for a row's sequence adds
    numbers of more than 31 bits."""
    n = (1 << 30) + 5
    table, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((n, 1), (n,)))
    start = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    table[-1], lens[-1], start[-1] = 1, 10, 4
    cache = M.Cache.empty(2, 1, 16, 64)
    cache.k.zero_()
    cache.v.zero_()
    seqs = M.Sequences(table, lens, start)
    k, v = (_q(4, 1, 64, s) for s in (51, 52))
    M.cache_write(cache, seqs, k, v)
    for x, y in ((cache.k, k), (cache.v, v)):
        assert not x[0].any() and not x[1, 0, :6].any() and not x[1, 0, 10:].any()
        assert torch.equal(x[1, 0, 6:10], y[:, 0])
    rk, rv = M.cache_read(cache, seqs, n=4)
    assert torch.equal(rk, k) and torch.equal(rv, v)


def test_a_threads_first_call():
    """A thread that has made no CUDA call before: nothing in the call itself relies on one."""
    import threading
    batch = Batch("bf16", [90, 30], None, 2, 64, 16, seed=61)
    q = _q(2, 4, 64, 62)
    want = M.attn_cached(batch.cache, batch.seqs, q)
    out = (torch.empty_like(q), torch.empty((4, 2), device="cuda"))
    ws = torch.empty(M.ATTN_CACHED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream()
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            M.attn_cached(batch.cache, batch.seqs, q, out=out, workspace=ws, stream=stream)
        except M.MarbleError as e:
            failed.append(e)

    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not failed, failed[0]
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("side", [False, True])
def test_threads_on_one_stream(side):
    """Calls with one workspace on one stream from several threads at once, as those on the same
    sequences are: a call's two kernels follow each other."""
    import ctypes
    import threading
    batch = Batch("bf16", [9000, 3000], None, 2, 64, 64, seed=61)
    qs = [_q(2, 8, 64, s) for s in range(62, 70)]
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    want = [M.attn_cached(batch.cache, batch.seqs, q) for q in qs]
    ws = torch.empty(M.ATTN_CACHED_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros((1000, *q.shape), dtype=torch.bfloat16, device="cuda") for q in qs]
    torch.cuda.synchronize()
    call, raw = M.lib().marble_attn_cached, stream.cuda_stream
    gate = threading.Barrier(len(qs))
    failed = []

    def work(q, out):
        descs = [M._AttnCached(q.data_ptr(), 512, o.data_ptr(), 512, None, 8, 0.0, M.WINDOW_INF, 0,
                               1, ws.data_ptr()) for o in out]
        descs = [ctypes.byref(d) for d in descs]
        gate.wait()
        for d in descs:
            if call(2, batch.cache._ref, batch.seqs._ref, d, None, raw) != M.OK:
                failed.append(M.lib().marble_last_error().decode())

    threads = [threading.Thread(target=work, args=a) for a in zip(qs, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[0]
    wrong = [int((out != w[0]).flatten(1).any(1).sum()) for out, w in zip(outs, want)]
    assert wrong == [0] * len(qs)
