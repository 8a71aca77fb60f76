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
