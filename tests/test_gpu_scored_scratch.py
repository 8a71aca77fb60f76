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
    """Grouped heads of few units have dK/dV of every q head in a scratch.  Where the cap leaves no
    room for it the backward runs without, as it does where the allocation fails."""
    n, hq, hkv, d, length = 8192, 32, 1, 128, 128
    tr = wl.tracks_from_samples([[wl.Span("causal", length)]] * (n // length))
    q, k, v, do = _qkvdo(n, hq, hkv, d, 41)
    slopes = _slopes(hq, "usual")
    pl = M.Plan(*device_tracks(tr), INF, 1)
    tiles, group = pl.stats()["nnz"] * hq * 32768, 8 * n * hq * d
    assert tiles < 100 << 20 < group
    score = M.Score(8.0, slopes)
    _run(pl, q, k, v, do, score, fused=True)  # torch's own buffers, and results with the scratch
    torch.cuda.synchronize()
    _capped(monkeypatch, 100)
    M.release_memory()
    before = torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved()
    got = _run(pl, q, k, v, do, score, fused=True)
    torch.cuda.synchronize()
    held = before - torch.cuda.mem_get_info()[0] - torch.cuda.memory_reserved()
    assert held < group  # the pool keeps what a call has freed
    for a in (0, 5 * length, n - length):
        cut = slice(a, a + length)
        sub = {x: np.asarray(tr[x])[cut] for x in ("sample", "seg", "noise")}
        part = (got[0][cut], got[1][:, cut]) + tuple(x[cut] for x in got[2:])
        _check(part, *(x[cut] for x in (q, k, v, do)), mask.dense_mask(sub, INF), 8.0, slopes)
