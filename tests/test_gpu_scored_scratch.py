"""The scored backward's scratch: what it does without room for it, against the fp64 oracle."""
import os

import numpy as np
import pytest
import torch

import context_attention_metadata_gb300 as M
import workloads as wl
from marble_testlib import device_tracks
from oracle import mask
from test_gpu_scored import INF, _check, _qkvdo, _run, _slopes

pytestmark = pytest.mark.gpu


def _capped(monkeypatch, mb):
    monkeypatch.setenv("MARBLE_DS_SCRATCH_CAP_MB", str(mb))


def test_grouped_heads_without_room_for_their_scratch(monkeypatch):
    """Grouped heads of long units have dK/dV of every q head in a scratch.  Where the cap leaves no
    room for it the backward runs without, as it does where the allocation fails."""
    hq, hkv, d, length, mb = 32, 1, 128, 1024, 100
    n = 4 * length
    tr = wl.tracks_from_samples([[wl.Span("causal", length)]] * 4)
    q, k, v, do = _qkvdo(n, hq, hkv, d, 41)
    slopes = _slopes(hq, "usual")
    pl = M.Plan(*device_tracks(tr), INF, 4)
    group = 8 * n * hq * d
    assert mb << 20 < group
    score = M.Score(8.0, slopes)

    def pool():  # what the library holds beside torch; its pool keeps what a call has freed
        torch.cuda.synchronize()
        return -torch.cuda.mem_get_info()[0] - torch.cuda.memory_reserved()

    _run(pl, q, k, v, do, score, fused=True)  # the plan's own scratch, kept from here on
    M.release_memory()
    start = pool()
    _run(pl, q, k, v, do, score, fused=True)
    assert pool() - start >= group
    _capped(monkeypatch, mb)
    M.release_memory()
    start = pool()
    got = _run(pl, q, k, v, do, score, fused=True)
    assert pool() - start < group
    for a in (0, n - length):
        cut = slice(a, a + length)
        sub = {x: np.asarray(tr[x])[cut] for x in ("sample", "seg", "noise")}
        part = (got[0][cut], got[1][:, cut]) + tuple(x[cut] for x in got[2:])
        _check(part, *(x[cut] for x in (q, k, v, do)), mask.dense_mask(sub, INF), 8.0, slopes)


@pytest.mark.parametrize("P,mb,hq,hkv,d", [(2, 4, 8, 2, 64), (4, 4, 8, 2, 64), (4, 12, 8, 2, 64),
                                           (4, 12, 6, 1, 128), (4, 14, 6, 1, 128), (2, 6, 4, 4, 128)])
def test_backward_outside_whole_rows(monkeypatch, P, mb, hq, hkv, d):
    """A scratch that does not hold the pack's dS tiles: the fused backward in ranges of every kv
    shard's ring, on side streams and in two buffers, with and without units of their own for a
    group's q heads; step lists in buffers of a few steps."""
    tr = wl.tracks_from_samples([[wl.Span("causal", 1200)], [wl.Span("full", 300),
                                                             wl.Span("causal", 548)]])
    n = len(tr["sample"])
    q, k, v, do = _qkvdo(n, hq, hkv, d, 42)
    slopes = _slopes(hq, "usual")
    pl = M.Plan(*device_tracks(tr), INF, P, "ptrr_block")
    assert pl.stats()["nnz"] * hq * 32768 > mb << 20
    _capped(monkeypatch, mb)
    score, m = M.Score(8.0, slopes), mask.dense_mask(tr, INF)
    for fused in (True, False):
        M.timing_enable(True)
        M.timing_read()
        got = _run(pl, q, k, v, do, score, fused=fused)
        launches = M.timing_read()["dkdv_launches"]
        M.timing_enable(False)
        assert launches > 1 if fused else launches > P
        _check(got, q, k, v, do, m, 8.0, slopes)
        again = [_run(pl, q, k, v, do, score, fused=fused),
                 _run(pl, q, k, v, do, score, fused=fused, stream=torch.cuda.Stream())]
        try:
            M.set_side_streams(0)
            again.append(_run(pl, q, k, v, do, score, fused=fused))
        finally:
            M.set_side_streams(4)
        for other in again:
            assert all(torch.equal(x, y) for x, y in zip(got, other))
