"""Paged caches for the tests, and what the kernels' roundings allow."""
import numpy as np
import torch

import context_attention_metadata_gb300 as M
from oracle import cached as C

U = 2.0 ** -24
HALF = {"bf16": torch.finfo(torch.bfloat16).eps / 2, "fp16": torch.finfo(torch.float16).eps / 2}
DTYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
E4M3 = C.e4m3_values()


def bf16(gen, shape, spread=0.5):
    """Heads of different sizes."""
    x = torch.randn(shape, generator=gen, device="cuda")
    s = torch.randn(shape[:-1] + (1,), generator=gen, device="cuda")
    return (x * torch.exp(spread * s)).bfloat16()


def np64(t):
    return t.detach().double().cpu().numpy()


def codes_of(t):
    """The values of a cache tensor, float64 on the host."""
    if t.dtype is torch.float8_e4m3fn:
        return E4M3[t.view(torch.uint8).cpu().numpy()]
    return np64(t)


def quantised(x, kind):
    """float64 heads [..., d] of bf16 values, finite -> (codes, scales): C.quantise_head for
    whole arrays.  x * 127 / top is rounded once, and no quotient of 15-bit numbers by 8-bit ones
    is nearer to a half than 2^-17, so float64 decides as rationals do."""
    top = np.abs(x).max(-1)
    safe = np.where(top == 0, 1, top)[..., None]
    if kind == "int8":
        return np.round(x * 127 / safe), (top.astype(np.float32) / np.float32(127)).astype(float)
    m, e = np.frexp(top)
    e = np.maximum(np.where(m <= 0.875, e - 9, e - 8), -126)
    s = np.ldexp(1.0, e)
    codes = torch.as_tensor(x / s[..., None]).to(torch.float8_e4m3fn).double().numpy()
    return codes, np.where(top == 0, 0.0, s)


class Batch:
    """Sequences of the given lengths in a pool of shuffled pages; what no sequence holds is
    poison: NaN values, codes and scales (int8: 127 with NaN scales)."""

    def __init__(self, kind, lens, counts, hkv, d, page, seed=0, spare=3, fill=True, stride_pad=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rng = np.random.default_rng(seed)
        lens = np.asarray(lens)
        need = -(-np.maximum(lens, 0) // page)
        pages = int(need.sum()) + spare
        self.kind, self.lens, self.page, self.hkv, self.d = kind, lens, page, hkv, d
        self.table = np.full((len(lens), max(1, int(need.max(initial=1)))), -7, np.int32)
        order = rng.permutation(pages)[:need.sum()]
        self.table[np.arange(self.table.shape[1]) < need[:, None]] = order
        self.start = None if counts is None else \
            np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.n = len(lens) if counts is None else int(np.sum(counts))
        self.pool = torch.empty((pages, 2 * hkv * page * d + stride_pad), dtype=DTYPES[kind],
                                device="cuda")
        if kind == "bf16":
            self.pool.fill_(float("nan"))
        else:
            self.pool.view(torch.int8).fill_(127)  # e4m3's NaN
        body = self.pool[:, :2 * hkv * page * d].unflatten(1, (2, hkv, page, d))
        self.scale = None
        if kind != "bf16":
            self.scale = torch.full((pages, 2, hkv, page), float("nan"), device="cuda")
        self.cache = M.Cache(body[:, 0], body[:, 1], *(
            (None, None) if self.scale is None else (self.scale[:, 0], self.scale[:, 1])))
        dev = lambda x: torch.as_tensor(np.asarray(x, np.int32)).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.seqs = M.Sequences(dev(self.table), dev(lens),
                                None if counts is None else dev(self.start), self.status)
        self.body = body
        self.k, self.v = [], []
        if fill:
            for b, length in enumerate(lens):
                x = np64(bf16(gen, (max(int(length), 0), 2, hkv, d)))
                if kind != "bf16" and length > 0:
                    codes, s = quantised(x, kind)
                    x = codes * s[..., None]
                else:
                    codes, s = x, None
                self.put(b, np.arange(max(int(length), 0)), codes, s)
                self.k.append(x[:, 0])
                self.v.append(x[:, 1])

    def put(self, b, pos, codes, scale):
        if len(pos) == 0:
            return
        g = torch.as_tensor(self.table[b][pos // self.page].astype(np.int64)).cuda()
        t = torch.as_tensor(pos % self.page).cuda()
        c = torch.as_tensor(codes).cuda()
        if self.kind == "e4m3":
            self.body.view(torch.int8)[g, :, :, t] = c.to(torch.float8_e4m3fn).view(torch.int8)
        else:
            self.body[g, :, :, t] = c.to(self.body.dtype)
        if scale is not None:
            self.scale[g, :, :, t] = torch.as_tensor(scale).float().cuda()

    def values(self):
        """(codes' values, scales) of the whole pool, [pages, 2, hkv, page, d] and without d."""
        return codes_of(self.body.contiguous()), None if self.scale is None else np64(self.scale)


def attn_bounds(ref, kind, d, keys, vmax, slopes=None, reach=0, cap=0.0):
    """(bound of |o - ref|, bound of |lse - ref|) by the kernel's roundings, u = 2^-24.
    A score: d products summed in fp32 (the matrix unit may cut instead of rounding: 2 u an
    addition of at most the terms' sum), 8 u more for the factors, the cap's tanh 4 u of the cap,
    the bias 3 u of itself.  A weight: that error, 8 u for exp2 and the maximum's subtraction,
    whose operands are at most the score; then its rounding, two bf16 terms (2^-16) or fp16
    (2^-11, and below its normal range 2^-25 / 64 of v's largest scale, which is at most twice
    vmax).  Sums over the keys: 2 u a key.  o is rounded to bf16 at the end."""
    bias = 0.0 if slopes is None else 3 * U * reach * np.abs(np.asarray(slopes))[:, None]
    e = (2 * d + 16) * U * ref["terms"] + 4 * U * cap + bias + 16 * U
    sums = 2 * U * (keys + 16)
    lse = e + sums + 4 * U * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0))
    w = 2.0 ** -16 if kind == "bf16" else HALF["fp16"]
    rel = (2 * e + w + 2 * sums).T[..., None]
    small = 0.0 if kind == "bf16" else keys * 2.0 ** -31 * 2 * vmax
    o = HALF["bf16"] * np.abs(ref["o"]) + (1 + HALF["bf16"]) * (rel * ref["abs"] + small)
    return o, lse


def check_attn(batch, q, o, lse, window=None, span=False, cap=0.0, slopes=None, scale=None):
    sl = None if slopes is None else np64(slopes)
    ref = C.attention(np64(q), batch.k, batch.v, batch.lens, batch.start, window, span, scale, cap,
                      sl)
    keys = int(max(batch.lens.max(initial=0), 1))
    vmax = max([np.abs(x).max() for x in batch.v if x.size] or [0.0])
    bo, bl = attn_bounds(ref, batch.kind, batch.d, keys, vmax, sl, keys, cap)
    n = ref["o"].shape[0]
    err = np.abs(np64(o)[:n] - ref["o"])
    assert (err <= bo).all(), (err - bo).max()
    got = np64(lse)
    assert (np.isneginf(got) == np.isneginf(ref["lse"])).all()
    live = np.isfinite(ref["lse"])
    err = np.abs(got[live] - ref["lse"][live])
    assert (err <= np.broadcast_to(bl, got.shape)[live]).all(), err.max()
