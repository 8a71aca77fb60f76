"""A chunk of a prompt behind its cached prefix, both ways: the whole sequences read into a pack's order
and the packed attention over them, with queries of zeros for the prefix's rows, and the cached
attention of the chunk's rows alone."""
import numpy as np
import pytest
import torch

import context_attention_metadata_gb300 as M
from cached_testlib import HALF, Batch, attn_bounds, bf16, check_attn, np64
from oracle import cached as C

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("window", [None, 100])
@pytest.mark.parametrize("d,shards,order", [(128, 4, "ptrr_block"), (64, 1, "contiguous")])
def test_a_chunk_behind_its_prefix(kind, window, d, shards, order):
    lens, new = np.array([300, 0, 517, 90, 64]), np.array([45, 0, 64, 90, 1])
    hq, hkv, n = 6, 2, 1024  # 971 rows in the pack, the others are a sample of their own
    batch = Batch(kind, lens, new, hkv, d, 16, seed=41)
    whole = np.concatenate([[0], np.cumsum(lens)])
    sample = torch.as_tensor(np.repeat(np.arange(6), [*lens, n - lens.sum()])).int().cuda()
    none = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    plan = M.Plan(sample, none, none, M.WINDOW_INF if window is None else window, shards, order)
    k, v = M.cache_read(batch.cache, M.Sequences(
        batch.seqs.table, batch.seqs.lens, torch.as_tensor(whole).int().cuda(), batch.status),
        plan=plan)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(42)
    q = bf16(gen, (int(new.sum()), hq, d))
    rows = torch.as_tensor(np.concatenate([np.arange(e - c, e) for e, c in zip(whole[1:], new)]))
    rows = rows.cuda()
    packed = torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda")
    packed[rows] = q
    o = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((hq, n), device="cuda")
    M.forward(plan, plan.permute(packed), k, v, M.State(n, hq, d), o, lse)
    plan.check()
    o = plan.permute(o, inverse=True)[rows]
    lse = lse[:, torch.argsort(plan.export("perm").long())][:, rows]
    # The packed call reads the cache's values rounded to bf16, and rounds a weight to bf16 before
    # its product with v (2^-8 of it); the sum takes it as it was.
    k, v = (np64(plan.permute(x, inverse=True)) for x in (k, v))
    split = lambda x: [x[a:b] for a, b in zip(whole[:-1], whole[1:])]
    ref = C.attention(np64(q), split(k), split(v), lens, batch.start, window)
    bo, bl = attn_bounds(ref, "bf16", d, int(lens.max()), np.abs(v).max())
    bo = bo + (1 + HALF["bf16"]) * HALF["bf16"] * ref["abs"]
    assert (np.abs(np64(o) - ref["o"]) <= bo).all()
    assert (np.abs(np64(lse) - ref["lse"]) <= bl).all()
    # the cached attention of the same rows
    oc, lc = M.attn_cached(batch.cache, batch.seqs, q,
                           window=M.WINDOW_INF if window is None else window)
    check_attn(batch, q, oc, lc, window)
    batch.seqs.check()
