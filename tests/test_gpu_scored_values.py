"""Small and large values under caps on both sides of where the forward does without a running
maximum: rows whose scores all are near -cap or near +cap, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import context_attention_metadata_gb300 as M
import workloads as wl
from marble_testlib import device_tracks
from oracle import mask, scored
from test_gpu_scored import HALF, INF, _np, _qkvdo, _slopes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [None, "usual"])
@pytest.mark.parametrize("cap", [30.0, 50.0, 55.0, 60.0])
@pytest.mark.parametrize("power", [-50, -36, 0, 30, 36])
def test_values_of_any_usual_size(power, cap, kind):
    n, d = 512, 64
    tr = wl.tracks_from_samples([[wl.Span("causal", 300), wl.Span("full", 212)]])
    q, k, v, _ = _qkvdo(n, 2, 1, d, 9)
    # scores of 4 caps in size, the sign of all of a row's alike
    k[..., 0] = 8.0
    sign = (-1.0) ** (torch.arange(n, device="cuda") // 7)
    q[..., 0] = (4 * cap / 8 * sign)[:, None]
    v *= 2.0 ** power
    slopes = _slopes(2, kind)
    pl = M.Plan(*device_tracks(tr), INF, 2)
    m = mask.dense_mask(tr, INF)
    st, o, lse = M.State(n, 2, d), torch.empty_like(q), torch.empty((2, n), device="cuda")
    ref = scored.attention(q, k, v, m, cap, None if slopes is None else _np(slopes), scale=1.0,
                           h=HALF)
    for fused in (False, True):
        M.forward(pl, q, k, v, st, o, lse, fused=fused, scale=1.0, score=M.Score(cap, slopes))
        pl.check()
        off = 2.0 ** -20 * cap + 2.0 ** -22 * n / 16  # the capped score's roundings, the bias's
        assert (np.abs(_np(lse) - ref["LSE"]) <= off + 2.0 ** -18).all()
        lim = (1 + HALF) * ((1 + 2 * off / HALF) * ref["bound"]["O"] + HALF * np.abs(ref["O"]))
        assert (np.abs(_np(o) - ref["O"]) <= lim).all()
