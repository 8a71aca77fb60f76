"""States of step lists that do not hold a row's own keys, with a cap and a bias: the same sums over
the keys seen so far as of any other list, against the fp64 oracle over those keys alone."""
import numpy as np
import pytest
import torch

import context_attention_metadata_gb300 as M
import workloads as wl
from marble_testlib import device_tracks
from oracle import mask, scored
from test_gpu_scored import HALF, INF, SOFT, _np, _qkvdo

pytestmark = pytest.mark.gpu

SHARDS = 4
LISTS = [[(3, 0)], [(3, 1), (3, 0)], [(2, 0)], [(3, 0), (3, 3)], [(3, 3), (3, 0)],
         [(3, 0), (3, 1), (3, 2), (3, 3)]]


@pytest.mark.parametrize("merge", ["carried", "fp32"])
@pytest.mark.parametrize("cap", [0.0, 50.0, 60.0])
@pytest.mark.parametrize("slope", [0.02, 0.5, 3.0])
def test_lists_without_the_own_shard(slope, cap, merge):
    n, hq, hkv, d = 1024, 4, 2, 64
    tr = wl.tracks_from_samples([[wl.Span("causal", 500), wl.Span("full", 100),
                                  wl.Span("causal", 424)]])
    pl = M.Plan(*device_tracks(tr), INF, SHARDS)
    q, k, v, _ = _qkvdo(n, hq, hkv, d, 21, scale=4.0)
    slopes = slope * torch.arange(1, hq + 1, device="cuda", dtype=torch.float32)
    full = mask.dense_mask(tr, INF)
    shard = np.arange(n) // (n // SHARDS)
    for steps in LISTS:
        r = steps[0][0]
        rows = shard == r
        m = full & np.isin(shard, [j for _, j in steps])[None, :]
        st = M.State(n, hq, d)
        st.o_acc.zero_(), st.m.fill_(float("-inf")), st.l.zero_()
        o, lse = torch.empty_like(q), torch.empty((hq, n), device="cuda")
        M.attn_steps(pl, q, k, v, [(r, j, i == 0) for i, (_, j) in enumerate(steps)], st,
                     merge=merge, score=M.Score(cap, slopes))
        M.attn_finalize(pl, st, o, lse)
        pl.check()
        ref = scored.attention(q, k, v, m, cap, _np(slopes), h=HALF)
        O, L = _np(o)[rows], _np(lse)[:, rows]
        assert m[rows].any(1).all() and np.isfinite(L).all()
        # scores of up to 60 and the bias of the list's farthest keys, of size S in all: the bias's
        # three roundings (slope, first key, sum), the score's, the LSE's three and two for every
        # merge, half a step each
        off = SOFT + (4 + len(steps)) * 2.0 ** -23 * (60 + float(slopes.max()) * n)
        assert (np.abs(L - ref["LSE"][:, rows]) <= off).all()
        # "fp32": every partial is rounded to fp32, and weighed by its LSE's rounding
        soft = 2 * len(steps) * off / HALF
        lim = (1 + HALF) * ((1 + soft) * ref["bound"]["O"] + HALF * np.abs(ref["O"]))
        assert (np.abs(O - ref["O"][rows]) <= lim[rows] + 1e-30).all()
        if merge == "carried":  # the state's own contract: sums of 2^(s - m) over these keys
            got = (st.m + torch.log2(st.l))[:, torch.as_tensor(rows)].double() * np.log(2)
            assert (np.abs(got.cpu().numpy() - ref["LSE"][:, rows]) <= off).all()
