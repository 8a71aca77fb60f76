"""What the cache operators are measured on: keys and values of new tokens written into a paged
cache (bf16, or quantised as they are written), read back out of it, and the attention of the next
tokens of a batch of sequences over it.

A case is a dict of plain values.  `prepare` makes its inputs from a seed, `run` is one pass of
the operator: in elementary torch operations, or, where `own` is true, by the library's calls.
`exact` gives the same outputs in 64 bits, `work` the bytes and operations of a pass.

The cache: pages of `page` tokens, [pages, hkv, page, d], keys and values of a page side by side
in one pool.  A sequence's position p is in page table[b, p // page], at p % page.  Quantised
types hold 8 bits a channel and one fp32 scale a token and head:
    e4m3: the smallest power of two that brings the head's largest channel to 448 or less,
    int8: the head's largest channel / 127.
"""
import math
import random

import numpy as np
import torch

own = False

BITS = {"bf16": 16, "e4m3": 8, "int8": 8}


# ----------------------------------------------------------------------------------- cases
def _cache(name, op, kind, seqs, past, new, hkv, d, page, shards, mix):
    """write: up to `new` tokens each of `seqs` sequences that hold up to `past`; append: the
    same, then the whole sequences read back; read: up to `new` tokens of each read.
    shards > 0: the tokens are in the order of a plan of so many shards."""
    return {"name": name, "op": op, "kind": kind, "seqs": seqs, "past": past, "new": new,
            "hkv": hkv, "d": d, "page": page, "shards": shards, "mix": mix}


def _attn(name, kind, seqs, past, new, hkv, group, d, page, window, cap, bias, span, mix):
    """Attention of up to `new` tokens each of `seqs` sequences, cached themselves, over up to
    `past` tokens before them.  window 0: none; cap 0: none; bias: a slope per head; span: the
    new tokens of a sequence all see each other."""
    return {"name": name, "op": "attn", "kind": kind, "seqs": seqs, "past": past, "new": new,
            "hkv": hkv, "group": group, "d": d, "page": page, "window": window, "cap": cap,
            "bias": bias, "span": span, "mix": mix}


def listed():
    return [
        # the next token of each of 32 sequences, written on its way to the attention
        _cache("write_step_32", "write", "e4m3", 32, 4096, 1, 8, 128, 64, 0, 1),
        # prompts of odd lengths, heads of 64
        _cache("write_prompts", "write", "bf16", 13, 0, 1500, 2, 64, 16, 0, 2),
        # the keys and values of a packed prefill of 256K tokens, in plan order
        _cache("write_pack_256k", "write", "e4m3", 24, 0, 20000, 8, 128, 64, 16, 3),
        # a chunk of a long prompt: written, then read with what was there before for the chunk's
        # own attention over a pack
        _cache("append_chunk", "append", "int8", 6, 14000, 2048, 8, 128, 128, 0, 4),
        # shared prefixes out of a small cache
        _cache("read_prefixes", "read", "e4m3", 9, 0, 777, 3, 64, 32, 0, 5),
        # one long sequence out of the cache
        _cache("read_long_256k", "read", "int8", 1, 0, 262144, 8, 128, 256, 0, 6),
        # the next token of one sequence: latency alone
        _attn("attn_one_2k", "bf16", 1, 2047, 1, 2, 1, 64, 64, 0, 0.0, False, False, 7),
        # the next token of one long sequence, heads as in the 256K configuration
        _attn("attn_one_256k", "bf16", 1, 262143, 1, 8, 4, 128, 64, 0, 0.0, False, False, 8),
        # a small batch with small pages and capped scores, seven q heads to a kv head
        _attn("attn_batch_61", "e4m3", 61, 4000, 1, 2, 7, 64, 16, 0, 30.0, False, False, 9),
        # a batch of sequences of all lengths in bf16
        _attn("attn_batch_64", "bf16", 64, 16384, 1, 8, 4, 128, 64, 0, 0.0, False, False, 10),
        # drafts checked in a window layer with a bias by distance
        _attn("attn_drafts_window", "int8", 40, 30000, 5, 8, 4, 128, 128, 4096, 0.0, True, False,
              11),
        # a large batch over an 8-bit cache
        _attn("attn_batch_128", "e4m3", 128, 16384, 1, 8, 8, 128, 64, 0, 0.0, False, False, 12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _most(op):
    return max(work(c)["bytes"] for c in listed() if c["op"] == op)


def _draw_cache(rng):
    op = rng.choice(("write", "append", "read"))
    kind = rng.choice(("bf16", "e4m3") if op == "write" else ("bf16", "e4m3", "int8"))
    new = _log_int(rng, 1, 20000)
    case = _cache("", op, kind, _log_int(rng, 1, 64), 0 if op == "read" else rng.choice(
        (0, _log_int(rng, 1, 16384))), new, rng.randint(1, 8), rng.choice((64, 128)),
        rng.choice((16, 32, 64, 128, 256)),
        rng.choice((0, 0, 4, 16)) if op == "write" and new > 64 else 0, rng.randrange(1 << 20))
    while work(case)["bytes"] > _most(op) or _padded(case) > 3e9:
        side = max(("seqs", "new", "past"), key=lambda x: case[x] * (64 if x == "seqs" else 1))
        case[side] = max(1, case[side] // 2)
    return case


def _draw_attn(rng):
    hkv = rng.choice((1, 2, 3, 4, 8))
    new = rng.choice((1, 1, 1, 2, 5, 8))
    cap, bias = rng.choice(((0, 0), (0, 0), (1, 0), (0, 1), (1, 1)))
    case = _attn("", rng.choice(("bf16", "e4m3", "int8")), _log_int(rng, 1, 256),
                 _log_int(rng, 1, 262144), new, hkv, rng.choice((1, 2, 4, 7, 8)),
                 rng.choice((64, 128)), rng.choice((16, 32, 64, 128, 256)),
                 rng.choice((0, 0, 0, 257, 4096)), rng.choice((20.0, 50.0)) if cap else 0.0,
                 bool(bias), new > 1 and rng.random() < 0.4, rng.randrange(1 << 20))
    while work(case)["bytes"] > _most("attn") or _padded(case) > 4.4e9:
        side = "seqs" if case["seqs"] > 8 and rng.random() < 0.5 else "past"
        case[side] = max(1, case[side] // 2)
    return case


def draw(rng):
    case = _draw_cache(rng) if rng.random() < 0.45 else _draw_attn(rng)
    del case["name"]
    return case


# -------------------------------------------------------------------------------- sequences
def _counts(case):
    """(new tokens, tokens held with them) of every sequence: all lengths up to the case's, the
    longest of each among them."""
    rng = np.random.default_rng(case["mix"])
    b = case["seqs"]
    new = rng.integers(1, case["new"] + 1, b)
    past = rng.integers(0, case["past"] + 1, b)
    new[rng.integers(0, b)] = case["new"]
    past[rng.integers(0, b)] = case["past"]
    return new, new + past


def _rows(case):
    """Rows of the token tensors: the new tokens, with a plan filled up to its whole blocks."""
    n = int(_counts(case)[0].sum())
    whole = 128 * case["shards"] if case.get("shards") else 1
    return -(-n // whole) * whole


def _padded(case):
    """Channels of keys and values if every sequence were as long as the longest."""
    return 2 * case["seqs"] * int(_counts(case)[1].max()) * case["hkv"] * case["d"]


def _first_seen(case, new, held):
    """The first position that any of a sequence's new tokens sees."""
    w = case["window"]
    return np.maximum(0, held - new - w + 1) if w else np.zeros_like(held)


def _deal(n, shards):
    """Token order of a causal pack dealt to the shards: blocks of 128, the costliest (the last)
    first, in rounds that turn at their ends; a shard keeps its blocks in sequence."""
    nb = n // 128
    i = np.arange(nb)
    rank = np.where(i // shards % 2 == 0, i % shards, shards - 1 - i % shards)
    of_block = np.empty(nb, np.int64)
    of_block[nb - 1 - i] = rank
    return (np.argsort(of_block, kind="stable")[:, None] * 128 + np.arange(128)).reshape(-1)


# ---------------------------------------------------------------------------------- inputs
def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    hkv, d, page, kind = case["hkv"], case["d"], case["page"], case["kind"]
    new, held = _counts(case)
    st = {"case": case}

    def normal(shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    def heads(*shape):  # tokens and heads of different sizes
        x = normal(shape + (d,))
        return x.mul_(normal(shape + (1,)).mul_(0.5).exp_())

    # pages in any order, one in sixteen of the pool unused, table entries behind a sequence's
    # last page -1
    need = -(-held // page)
    pages = int(need.sum()) + int(need.sum()) // 16 + 1
    table = np.full((len(held), int(need.max())), -1, np.int32)
    table[np.arange(table.shape[1]) < need[:, None]] = rng.permutation(pages)[:need.sum()]
    st["table"] = torch.as_tensor(table).cuda()
    st["held"] = torch.as_tensor(held.astype(np.int32)).cuda()
    st["start"] = torch.as_tensor(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    shape = (pages, 2, hkv, page)
    if case["op"] == "write":  # what was there before does not matter
        st["pool"] = torch.zeros(shape + (d,), device="cuda",
                                 dtype=torch.bfloat16 if kind == "bf16" else torch.int8)
        st["scale"] = None if kind == "bf16" else torch.zeros(shape, device="cuda")
    else:
        st["pool"], st["scale"] = _quantised(heads(*shape), kind)
    if case["op"] in ("write", "append"):  # a projection's output
        n = _rows(case)
        st["kv"] = heads(n, 2 * hkv)
        st["n"] = n
    if case["op"] == "append":
        st["whole"] = torch.as_tensor(np.concatenate([[0], np.cumsum(held)]).astype(np.int32))
        st["whole"] = st["whole"].cuda()
    if case["op"] == "attn":
        hq = hkv * case["group"]
        # scores with a standard deviation of 2.5
        st["q"] = normal((int(new.sum()), hq, d)).mul_(2.5)
        st["slopes"] = None
        if case["bias"]:
            st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)],
                                        dtype=torch.float32, device="cuda")
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["perm"] = None
    if case.get("shards"):
        st["perm"] = torch.as_tensor(_deal(st["n"], case["shards"])).cuda()
    if case["op"] == "attn":
        st["out"] = (torch.empty_like(st["q"]),
                     torch.empty((st["q"].shape[1], st["q"].shape[0]), device="cuda"))
    elif case["op"] != "write":
        n = int(_counts(case)[case["op"] == "append"].sum())
        st["out"] = torch.empty((n, 2 * case["hkv"], case["d"]), dtype=torch.bfloat16,
                                device="cuda")
    if own:
        import context_attention_metadata_gb300 as M
        st["M"] = M
        pool, scale = st["pool"], st["scale"]
        if case["kind"] == "e4m3":
            pool = pool.view(torch.float8_e4m3fn)
        st["cache"] = M.Cache(pool[:, 0], pool[:, 1], *(
            (None, None) if scale is None else (scale[:, 0], scale[:, 1])))
        one = case["new"] == 1
        st["seqs"] = M.Sequences(st["table"], st["held"], None if one else st["start"])
        st["plan"] = None
        if case["op"] == "append":
            st["all"] = M.Sequences(st["table"], st["held"], st["whole"])
        if case.get("shards"):
            n = st["n"]
            zero = torch.zeros(n, dtype=torch.int32, device="cuda")
            none = torch.full((n,), -1, dtype=torch.int32, device="cuda")
            st["plan"] = M.Plan(zero, none, none, M.WINDOW_INF, case["shards"], "ptrr_block")
        if case["op"] == "attn":
            st["score"] = M.Score(cap=case["cap"], slopes=st["slopes"]) \
                if case["cap"] or case["bias"] else None
    return st


# ------------------------------------------------------------------------------------- run
def run(st):
    op = st["case"]["op"]
    if own:
        return {"write": _own_write, "append": _own_append, "read": _own_read,
                "attn": _own_attn}[op](st)
    return {"write": _plain_write, "append": _plain_append, "read": _plain_read,
            "attn": _plain_attn}[op](st)


def _state(st):
    """The cache's pool as the values it holds, and the scales."""
    if st["case"]["kind"] == "bf16":
        return (st["pool"],)
    return st["pool"].view(torch.float8_e4m3fn), st["scale"]


def _own_write(st):
    k, v = st["kv"].split(st["case"]["hkv"], dim=1)
    st["M"].cache_write(st["cache"], st["seqs"], k, v, plan=st["plan"])
    return _state(st)


def _own_append(st):
    h = st["case"]["hkv"]
    k, v = st["kv"].split(h, dim=1)
    st["M"].cache_write(st["cache"], st["seqs"], k, v)
    st["M"].cache_read(st["cache"], st["all"], out=st["out"].split(h, dim=1))
    return st["out"]


def _own_read(st):
    st["M"].cache_read(st["cache"], st["seqs"], out=st["out"].split(st["case"]["hkv"], dim=1))
    return st["out"]


def _own_attn(st):
    c, M = st["case"], st["M"]
    return M.attn_cached(st["cache"], st["seqs"], st["q"], window=c["window"] or M.WINDOW_INF,
                         span=c["span"], score=st["score"], new_tokens=c["new"], out=st["out"])


def _quantised(x, kind):
    """bf16 heads [..., d] -> (codes, scales [...] or None); the codes of e4m3 as int8 bits."""
    if kind == "bf16":
        return x, None
    x = x.float()
    top = x.abs().amax(-1, keepdim=True)
    if kind == "e4m3":
        m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
        scale = torch.ldexp(torch.ones_like(top), torch.where(m <= 0.875, e - 9, e - 8))
        scale = torch.where(top == 0, torch.zeros_like(top), scale)
        codes = (x / torch.where(top == 0, torch.ones_like(top), scale)) \
            .to(torch.float8_e4m3fn).view(torch.int8)
    else:
        # x * 127 is exact, and its quotient is no nearer to a half than fp32 can tell
        scale = top / 127
        codes = (x * 127 / torch.where(top == 0, torch.ones_like(top), top)).round()
        codes = codes.to(torch.int8)
    return codes, scale.squeeze(-1)


def _values(codes, scale, kind):
    """What the codes stand for, fp32."""
    if kind == "bf16":
        return codes.float()
    x = codes.view(torch.float8_e4m3fn).float() if kind == "e4m3" else codes.float()
    return x * scale[..., None]


def _places(st, start):
    """(sequence, position) of every row below start[-1]."""
    n = int(_counts(st["case"])[0 if start is st["start"] else 1].sum())
    row = torch.arange(n, device="cuda")
    seq = torch.searchsorted(start[1:].long(), row, right=True)
    return seq, st["held"].long()[seq] - (start[seq + 1] - row)


def _plain_write(st):
    c = st["case"]
    h, n = c["hkv"], int(_counts(c)[0].sum())
    kv = st["kv"]
    if st["perm"] is not None:  # back to the order of the sequences
        back = torch.empty_like(kv)
        back[st["perm"]] = kv
        kv = back
    codes, scale = _quantised(kv[:n].view(n, 2, h, c["d"]), c["kind"])
    seq, pos = _places(st, st["start"])
    page, slot = st["table"].long()[seq, pos // c["page"]], pos % c["page"]
    st["pool"][page, :, :, slot] = codes
    if scale is not None:
        st["scale"][page, :, :, slot] = scale
    return _state(st) if c["op"] == "write" else None


def _plain_out(st, start):
    c = st["case"]
    seq, pos = _places(st, start)
    page, slot = st["table"].long()[seq, pos // c["page"]], pos % c["page"]
    scale = None if st["scale"] is None else st["scale"][page, :, :, slot]
    x = _values(st["pool"][page, :, :, slot], scale, c["kind"])
    return x.bfloat16().view(-1, 2 * c["hkv"], c["d"])


def _plain_append(st):
    _plain_write(st)
    return _plain_out(st, st["whole"])


def _plain_read(st):
    return _plain_out(st, st["start"])


def _plain_attn(st):
    """Every sequence padded to the longest, its new tokens to the most."""
    c = st["case"]
    b, new, h, g, d = c["seqs"], c["new"], c["hkv"], c["group"], c["d"]
    n = st["q"].shape[0]
    table = st["table"].long().clamp(min=0)
    length = table.shape[1] * c["page"]

    def whole(which):  # [b, h, length, d]
        codes = st["pool"][:, which][table]
        scale = None if st["scale"] is None else st["scale"][:, which][table]
        return _values(codes, scale, c["kind"]).transpose(1, 2).reshape(b, h, length, d)

    seq, pos = _places(st, st["start"])
    at = torch.arange(n, device="cuda") - st["start"].long()[seq]
    q = torch.zeros((b, new, h, g, d), device="cuda")
    q[seq, at] = st["q"].float().view(n, h, g, d)
    where = torch.full((b, new), -1, device="cuda")
    where[seq, at] = pos
    key = torch.arange(length, device="cuda")
    far = where[:, :, None] - key  # [b, new, length]
    see = (far >= 0) & (far < (c["window"] or length + 1))
    held, count = st["held"].long(), (st["start"][1:] - st["start"][:-1]).long()
    if c["span"]:
        see |= ((key >= (held - count)[:, None]) & (key < held[:, None]))[:, None]
    s = q.permute(0, 2, 1, 3, 4).reshape(b, h, new * g, d) @ whole(0).transpose(-1, -2)
    s = s.view(b, h, new, g, length) * (1.0 / math.sqrt(d))
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    if st["slopes"] is not None:
        s = s - st["slopes"].view(h, 1, g, 1) * far.abs()[:, None, :, None]
    s = s.masked_fill(~see[:, None, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    v = whole(1).masked_fill((key >= held[:, None])[:, None, :, None], 0.0)
    o = (p / total).view(b, h, new * g, length) @ v
    o = o.view(b, h, new, g, d).permute(0, 2, 1, 3, 4)[seq, at].reshape(n, h * g, d)
    lse = (m + total.log()).view(b, h, new, g).permute(0, 2, 1, 3)[seq, at].reshape(n, h * g)
    return o.bfloat16(), lse.t().contiguous()


# ----------------------------------------------------------------------------------- exact
def exact(case, seed):
    st = _inputs(case, seed)
    return {"write": _exact_write, "append": _exact_out, "read": _exact_out,
            "attn": _exact_attn}[case["op"]](case, st)


def _power(x):
    """The power of two at or below each of x > 0: its exponent bits."""
    return (x.view(torch.int64) >> 52 << 52).view(torch.float64)


def _exact_quantised(x, kind):
    """(values of the codes, scales) of heads in 64 bits."""
    x = x.double()
    if kind == "bf16":
        return x, None
    top = x.abs().max(-1).values
    if kind == "int8":
        return torch.round(x * 127 / top[..., None]), top / 127
    scale = _power(top / 448)
    scale = torch.where(top > 448 * scale, 2 * scale, scale)
    y = x / scale[..., None]
    # four significant bits down to 2^-6, steps of 2^-9 below
    step = _power(y.abs().clamp(min=2.0 ** -6)) / 8
    return torch.round(y / step) * step, scale


def _exact_sequence(case, st, b):
    """(codes' values, scales) [held, 2, hkv, d] of a sequence's cached tokens, 64 bits."""
    held = int(_counts(case)[1][b])
    pages = st["table"][b, :-(-held // case["page"])].long()
    x = st["pool"][pages].transpose(1, 3).flatten(0, 1)[:held].transpose(1, 2)
    if case["kind"] == "bf16":
        return x.double(), None
    s = st["scale"][pages].permute(0, 3, 1, 2).flatten(0, 1)[:held]
    return (x.view(torch.float8_e4m3fn) if case["kind"] == "e4m3" else x).double(), s.double()


def _exact_rows(case, st):
    """The new tokens in the order of the sequences, [n, 2, hkv, d]."""
    n = int(_counts(case)[0].sum())
    kv = st["kv"]
    if case["shards"]:
        kv = kv[torch.as_tensor(np.argsort(_deal(st["n"], case["shards"]))).cuda()]
    return kv[:n].unflatten(1, (2, case["hkv"]))


def _exact_write(case, st):
    new, held = _counts(case)
    values, scales = _exact_quantised(_exact_rows(case, st), case["kind"])
    pool = torch.zeros(st["pool"].shape, dtype=torch.float64, device="cuda")
    scale = torch.zeros(st["pool"].shape[:-1], dtype=torch.float64, device="cuda")
    table, at = st["table"].cpu().numpy(), 0
    for b in range(case["seqs"]):
        p = np.arange(held[b] - new[b], held[b])
        page = torch.as_tensor(table[b, p // case["page"]].astype(np.int64)).cuda()
        slot = torch.as_tensor(p % case["page"]).cuda()
        pool[page, :, :, slot] = values[at:at + new[b]]
        if scales is not None:
            scale[page, :, :, slot] = scales[at:at + new[b]]
        at += new[b]
    return (pool,) if scales is None else (pool, scale)


def _exact_out(case, st):
    new, held = _counts(case)
    out, at = [], 0
    if case["op"] == "append":
        written, scales = _exact_quantised(_exact_rows(case, st), case["kind"])
        if scales is not None:
            written = written * scales[..., None]
    for b in range(case["seqs"]):
        x, s = _exact_sequence(case, st, b)
        x = x if s is None else x * s[..., None]
        if case["op"] == "append":
            x = torch.cat((x[:held[b] - new[b]], written[at:at + new[b]]))
            at += new[b]
        else:
            x = x[held[b] - new[b]:]
        out.append(x.flatten(1, 2))
    return torch.cat(out)


def _exact_attn(case, st):
    """Sequence by sequence, token by token."""
    new, held = _counts(case)
    h, g, d = case["hkv"], case["group"], case["d"]
    q = st["q"].double()
    o = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty((h * g, q.shape[0]), dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["seqs"]):
        x, scale = _exact_sequence(case, st, b)
        x = x if scale is None else x * scale[..., None]
        k, v = x[:, 0].transpose(0, 1), x[:, 1].transpose(0, 1)  # [hkv, held, d]
        for t in range(new[b]):
            p = int(held[b] - new[b] + t)
            lo = max(0, p - case["window"] + 1) if case["window"] else 0
            hi = p + 1
            if case["span"]:
                lo, hi = min(lo, int(held[b] - new[b])), int(held[b])
            s = torch.einsum("hgd,hkd->hgk", q[at].view(h, g, d), k[:, lo:hi]) / d ** 0.5
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            if case["bias"]:
                ago = (p - torch.arange(lo, hi, device="cuda")).abs()
                s = s - st["slopes"].double().view(h, g, 1) * ago
            o[at] = (torch.softmax(s, -1) @ v[:, lo:hi]).view(h * g, d)
            lse[:, at] = torch.logsumexp(s, -1).view(-1)
            at += 1
    return o, lse


# ------------------------------------------------------------------------------------ work
def work(case):
    new, held = _counts(case)
    n, h, d = int(new.sum()), case["hkv"], case["d"]
    row = 2 * h * (d * BITS[case["kind"]] // 8 + (0 if case["kind"] == "bf16" else 4))
    if case["op"] == "attn":  # every key and value that some new token sees, q in, o and lse out
        hq = h * case["group"]
        keys = int((held - _first_seen(case, new, held)).sum())
        pairs = 0
        for count, m in zip(new, held):
            p = np.arange(m - count, m)
            lo = np.maximum(0, p - case["window"] + 1) if case["window"] else 0 * p
            pairs += int(((m if case["span"] else p + 1) - np.minimum(lo, m - count)
                          if case["span"] else p + 1 - lo).sum())
        return {"bytes": keys * row + n * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}
    token = 2 * h * d * 2
    if case["op"] == "append":
        whole = int(held.sum())
        return {"bytes": n * (token + row) + whole * (token + row), "flops": 3 * (n + whole) * h * d}
    return {"bytes": n * (token + row), "flops": 3 * n * h * d}
