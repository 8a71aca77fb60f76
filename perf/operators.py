"""What the rotary and the scored-attention operators are measured on: rotary positions with
several axes (with the heads' RMS norm, moved into plan order) and their gradient; attention over
a packed mask whose scores are capped by a tanh or get a bias by distance, and its gradients.

A case is a dict of plain values.  `prepare` makes its inputs from a seed, `run` is one pass of
the operator: in elementary torch operations, or, where `own` is true, by the library's calls.
`exact` gives the same outputs in 64 bits, `work` the bytes and operations of a pass.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 10000.0
PAIRINGS = ("halves", "adjacent")
LAYOUTS = ("sections", "axial", "interleaved")


# ----------------------------------------------------------------------------------- cases
def _rope(name, grad, n, hq, hkv, d, rot, axes, layout, pairing, norm, shards):
    """shards > 0: a causal pack of n tokens dealt to that many shards; 0: tokens as they are."""
    return {"name": name, "op": "rope_grad" if grad else "rope", "n": n, "hq": hq, "hkv": hkv,
            "d": d, "rot": rot, "axes": axes, "layout": layout, "pairing": pairing, "norm": norm,
            "shards": shards}


def _attn(name, train, n, hq, hkv, d, pack, window, cap, bias, shards, pack_seed):
    """window 0: none; cap 0: none; bias: a slope per head."""
    return {"name": name, "op": "attn_train" if train else "attn", "n": n, "hq": hq, "hkv": hkv,
            "d": d, "pack": pack, "window": window, "cap": cap, "bias": bias, "shards": shards,
            "pack_seed": pack_seed}


def listed():
    return [
        # the next token of one sequence: latency alone
        _rope("rope_one_token", False, 1, 32, 8, 128, 128, 3, "sections", "halves", True, 0),
        # the next tokens of a batch, a model that rotates half of each head
        _rope("rope_batch_61", False, 61, 14, 2, 64, 32, 1, "axial", "adjacent", False, 0),
        # the tiny packed configuration: text, an image, text
        _rope("rope_pack_2k", False, 2048, 2, 2, 64, 64, 3, "interleaved", "halves", False, 4),
        # every q, k and v of the 256K configuration, into plan order
        _rope("rope_pack_256k", False, 262144, 32, 8, 128, 128, 3, "sections", "halves", True, 16),
        # the gradient of an image batch of odd length, not packed
        _rope("rope_grad_5003", True, 5003, 12, 3, 64, 64, 2, "axial", "halves", True, 0),
        # the gradients of the 256K configuration, out of plan order
        _rope("rope_grad_pack_256k", True, 262144, 32, 8, 128, 128, 3, "sections", "halves", True,
              16),
        # the tiny packed configuration with capped scores
        _attn("attn_cap_2k", False, 2048, 2, 2, 64, "image", 0, 30.0, False, 4, 1),
        # a window layer with a bias by distance and grouped heads
        _attn("attn_bias_window_16k", False, 16384, 32, 8, 128, "causal", 4096, 0.0, True, 16, 2),
        # the 64K packed configuration with capped scores
        _attn("attn_cap_mix_64k", False, 65536, 16, 16, 128, "mix", 0, 50.0, False, 8, 3),
        # a training pass of a small pack with both, grouped heads, samples of odd lengths
        _attn("attn_train_both_4k", True, 4096, 8, 2, 64, "mix", 0, 30.0, True, 4, 4),
        # a training pass over image groups with a bias by distance
        _attn("attn_train_bias_16k", True, 16384, 8, 8, 128, "group", 0, 0.0, True, 8, 5),
        # a training pass of the 64K packed configuration with capped scores
        _attn("attn_train_cap_64k", True, 65536, 16, 16, 128, "mix", 0, 50.0, False, 8, 3),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rope(rng):
    d = rng.choice((64, 128))
    hkv = rng.randint(1, 8)
    hq = hkv * rng.choice((1, 2, 3, 4, 7))
    axes = rng.randint(1, 4)
    rot = 16 * rng.randint(1, d // 16)
    top = min(262144, 262144 * 48 * 128 // ((hq + 2 * hkv) * d))
    shards = rng.choice((0, 0, 1, 4, 8, 16))
    n = _log_int(rng, 1, top)
    if shards:
        n = max(1, n // (128 * shards)) * 128 * shards
    return _rope("", rng.random() < 0.5, n, hq, hkv, d, rot, axes, rng.choice(LAYOUTS),
                 rng.choice(PAIRINGS), rng.random() < 0.6, shards)


def _draw_attn(rng):
    d = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 3, 4, 8))
    hq = hkv * rng.choice((1, 2, 4))
    shards = rng.choice((1, 2, 4, 8))
    blocks = _log_int(rng, 1, 512) // shards * shards or shards
    pack = rng.choice(("mix", "group", "image", "causal"))
    cap, bias = rng.choice(((1, 0), (0, 1), (1, 1)))
    case = _attn("", rng.random() < 0.5, 128 * blocks, hq, hkv, d, pack,
                 rng.choice((0, 0, 257, 2048)) if pack == "causal" else 0,
                 rng.choice((15.0, 20.0, 30.0, 50.0)) if cap else 0.0, bool(bias), shards,
                 rng.randrange(1 << 20))
    most = max(work(c)["flops"] for c in listed() if c["op"] == case["op"])
    while work(case)["flops"] > most:  # one long sample: its pairs grow with the square
        case["n"] = max(1, case["n"] // (256 * shards)) * 128 * shards
    return case


def draw(rng):
    case = _draw_rope(rng) if rng.random() < 0.5 else _draw_attn(rng)
    del case["name"]
    return case


# ----------------------------------------------------------------------------------- packs
def _spans(case):
    """The pack as samples of (kind, length) spans; the last sample is the padding that fills it
    to whole blocks, odd lengths before it."""
    rng = random.Random(case["pack_seed"])
    n, kind, out, total = case["n"], case["pack"], [], 0
    real = n - rng.randint(0, 127)
    if kind == "causal":
        out = [[("causal", real)]]
    elif kind == "image":  # text, an image, text
        a, c = max(1, real * 3 // 8), max(1, real // 8)
        out = [[("causal", a)], [("full", real - a - c)], [("causal", c)]]
    while kind in ("mix", "group") and total < real:
        text = min(16384, max(16, round(rng.lognormvariate(math.log(650.0), 1.5))))
        image = rng.randint(256, 4096)
        u = rng.random()
        if kind == "group":  # text, then images of one group with text between
            s = [("causal", rng.randint(256, 2048))]
            s += [x for _ in range(rng.randint(2, 4))
                  for x in (("group", 1024), ("causal", rng.randint(64, 512)))]
        elif u < 0.6:
            s = [("causal", text)]
        elif u < 0.9:
            s = [("full", image), ("causal", text)]
        else:
            s = [("causal", text), ("noise", image), ("causal", max(16, text // 4))]
        cut = []
        for m, length in s:
            length = min(length, real - total)
            if length > 0:
                cut.append((m, length))
                total += length
        out.append(cut)
    if real < n:
        out.append([("causal", n - real)])
    return out


def _tracks(case):
    """sample, segment and noise ids of every token (int32, host)."""
    sample, seg, noise, nid = [], [], [], 0
    for i, s in enumerate(_spans(case)):
        group = None
        for m, length in s:
            g = z = -1
            if m == "group" and group is not None:
                g = group
            elif m != "causal":
                g, nid = nid, nid + 1
            if m == "group":
                group = g
            if m == "noise":
                z = g
            sample.append(np.full(length, i, np.int32))
            seg.append(np.full(length, g, np.int32))
            noise.append(np.full(length, z, np.int32))
    return tuple(np.concatenate(x) for x in (sample, seg, noise))


def _pairs(case):
    """Pairs of a query and a key that it may see, per head."""
    w = case["window"] or case["n"]
    total = 0
    for s in _spans(case):
        start, at = [], 0
        for _, length in s:
            start.append(at)
            at += length
        for i, (mi, li) in enumerate(s):
            if mi == "causal" and w < at:
                # query t of the span: the keys (t - w, t] of the sample outside noise spans
                hidden = np.zeros(at + 1, np.int64)
                for j, (mj, lj) in enumerate(s):
                    if mj == "noise":
                        hidden[start[j] + 1:start[j] + lj + 1] = 1
                hidden = np.cumsum(hidden)
                t = np.arange(start[i], start[i] + li)
                a = np.maximum(0, t - w + 1)
                total += int((t + 1 - a - (hidden[t + 1] - hidden[a])).sum())
                continue
            for j, (mj, lj) in enumerate(s):
                if i == j:
                    total += li * (li + 1) // 2 if mi == "causal" else li * li
                elif mi == mj == "group" or (j < i and mj != "noise"):
                    total += li * lj
    return total


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
def _sections(case):
    """Rotated pairs per axis: an equal share each, what is left to the first."""
    pairs, axes = case["rot"] // 2, case["axes"]
    share = pairs // axes
    return [pairs - share * (axes - 1)] + [share] * (axes - 1)


def _frequencies(case):
    """(radians per position, axis) of every rotated pair."""
    sections = _sections(case)
    pairs = sum(sections)
    i = np.arange(pairs)
    axis = np.repeat(np.arange(len(sections)), sections)
    if case["layout"] == "axial":  # a sequence of its own for every axis
        inside = np.concatenate([np.arange(s) / max(s, 1) for s in sections])
        return THETA ** -inside, axis
    if case["layout"] == "interleaved":  # the axes take turns while their pairs last
        turn = np.concatenate([np.arange(s) for s in sections])
        axis = axis[np.lexsort((axis, turn))]
    return THETA ** -(i / pairs), axis


def _positions(case, rng):
    """int32 [axes, n]: text and patches of images, as a packed sequence or a batch has them."""
    n, axes = case["n"], case["axes"]
    if n < 128:  # the next tokens of sequences of different lengths
        return rng.integers(0, 1 << 17, (1, n)).repeat(axes, 0).astype(np.int32)
    pos = np.tile(np.arange(n), (axes, 1))
    side = int(rng.integers(16, 65))
    first = int(rng.integers(0, n // 4))
    m = n // 2  # half of the sequence: frames of side x side patches
    j = np.arange(m)
    grid = [first + j // (side * side), first + j // side % side, first + j % side]
    for a in range(min(axes, 3) if axes > 1 else 0):
        pos[a, first:first + m] = grid[a if axes > 2 else a + 1]
    return pos.astype(np.int32)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]

    def normal(shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    st = {"case": case}
    if case["op"].startswith("rope"):
        rng = np.random.default_rng(seed)
        st["pos"] = torch.as_tensor(_positions(case, rng)).cuda()
        st["qkv"] = normal((n, hq + 2 * hkv, d), scale=1.5)  # a projection's output
        st["wq"], st["wk"] = ((1 + normal((d,), torch.float32, 0.2)) if case["norm"] else None
                              for _ in range(2))
        if case["op"] == "rope_grad":  # gradients in plan order
            st["dq"], st["dk"], st["dv"] = (normal((n, h, d), torch.float32)
                                            for h in (hq, hkv, hkv))
        return st
    # scores with a standard deviation of 2.5, some of them near the cap
    st["q"], st["k"], st["v"] = normal((n, hq, d), scale=2.5), normal((n, hkv, d)), \
        normal((n, hkv, d))
    if case["op"] == "attn_train":
        st["do"] = normal((n, hq, d))
    st["sample"], st["seg"], st["noise"] = (torch.as_tensor(x).cuda() for x in _tracks(case))
    st["slopes"] = None
    if case["bias"]:
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)],
                                    dtype=torch.float32, device="cuda")
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
    if case["op"].startswith("rope"):
        st["perm"] = None
        if case["shards"]:
            st["perm"] = torch.as_tensor(_deal(n, case["shards"])).cuda()
        freq, axis = _frequencies(case)
        st["freq"], st["axis"] = torch.as_tensor(freq).cuda(), torch.as_tensor(axis).cuda()
        if own:
            import context_attention_metadata_gb300 as M
            st["M"] = M
            st["rope"] = M.Rope(freq, axis, pairing=case["pairing"])
            st["plan"] = None
            if case["shards"]:
                zero = torch.zeros(n, dtype=torch.int32, device="cuda")
                none = torch.full((n,), -1, dtype=torch.int32, device="cuda")
                st["plan"] = M.Plan(zero, none, none, M.WINDOW_INF, case["shards"], "ptrr_block")
        return st
    sample = st["sample"].cpu().numpy()
    change = np.flatnonzero(np.diff(sample)) + 1
    bounds = np.concatenate([[0], change, [n]])
    st["first"] = bounds[sample]     # of each token's sample
    st["last"] = bounds[sample + 1]
    if own:
        import context_attention_metadata_gb300 as M
        st["M"] = M
        st["plan"] = M.Plan(st["sample"], st["seg"], st["noise"], case["window"] or M.WINDOW_INF,
                            case["shards"], "contiguous")
        st["state"] = M.State(n, hq, d)
        st["score"] = M.Score(cap=case["cap"], slopes=st["slopes"])
        st["grad"] = torch.empty(n * (hq + 2 * hkv) * d, device="cuda") \
            if case["op"] == "attn_train" else None
    return st


# ------------------------------------------------------------------------------------- run
def run(st):
    op = st["case"]["op"]
    if own:
        return {"rope": _own_rope, "rope_grad": _own_rope_grad, "attn": _own_attn,
                "attn_train": _own_attn}[op](st)
    return {"rope": _plain_rope, "rope_grad": _plain_rope_grad, "attn": _plain_attn,
            "attn_train": _plain_attn}[op](st)


def _split(st):
    c = st["case"]
    return st["qkv"].split((c["hq"], c["hkv"], c["hkv"]), dim=1)


def _own_rope(st):
    q, k, v = _split(st)
    return st["M"].rope(st["rope"], st["pos"], q, k, v, plan=st["plan"], q_weight=st["wq"],
                        k_weight=st["wk"], eps=EPS)


def _own_rope_grad(st):
    c = st["case"]
    q, k, _ = _split(st)
    out = torch.empty_like(st["qkv"])
    dq, dk, dv, dwq, dwk = st["M"].rope_bwd(
        st["rope"], st["pos"], st["dq"], st["dk"], st["dv"], plan=st["plan"], q=q, k=k,
        q_weight=st["wq"], k_weight=st["wk"], eps=EPS,
        out=out.split((c["hq"], c["hkv"], c["hkv"]), dim=1))
    return (out, dwq, dwk) if c["norm"] else (out,)


def _own_attn(st):
    M, c, plan = st["M"], st["case"], st["plan"]
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    q, k, v = st["q"], st["k"], st["v"]
    o = torch.empty_like(q)
    lse = torch.empty((hq, n), dtype=torch.float32, device="cuda")
    M.forward(plan, q, k, v, st["state"], o, lse, fused=True, score=st["score"])
    if c["op"] == "attn":
        return o, lse
    acc = st["grad"].zero_()
    dq, dk, dv = (x.view(n, h, d) for x, h in zip(
        acc.split((n * hq * d, n * hkv * d, n * hkv * d)), (hq, hkv, hkv)))
    delta = torch.empty_like(lse)
    M.backward(plan, q, k, v, o, st["do"], lse, delta, dq, dk, dv, fused=True, score=st["score"])
    grad = torch.empty(acc.shape, dtype=torch.bfloat16, device="cuda")
    M.cast_bf16(acc, grad)
    gq, gk, gv = grad.split((n * hq * d, n * hkv * d, n * hkv * d))
    return o, lse, gq.view(n, hq, d), gk.view(n, hkv, d), gv.view(n, hkv, d)


def _angles(st):
    """cos and sin [n, 1, pairs] of every token: the angles in 64 bits."""
    a = st["pos"].double()[st["axis"]].t() * st["freq"]
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _pair_up(x, case):
    """The rotated channels of x as (first, second) of every pair, and the rest."""
    rot = case["rot"]
    if case["pairing"] == "halves":
        return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]
    return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]


def _put_back(a, b, rest, case):
    if case["pairing"] == "halves":
        return torch.cat((a, b, rest), -1)
    return torch.cat((torch.stack((a, b), -1).flatten(-2), rest), -1)


def _plain_rope(st):
    case = st["case"]
    cos, sin = _angles(st)

    def move(x):
        return x.bfloat16() if st["perm"] is None else x.bfloat16()[st["perm"]]

    def turn(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        a, b, rest = _pair_up(x, case)
        return move(_put_back(a * cos - b * sin, a * sin + b * cos, rest, case))

    q, k, v = _split(st)
    return turn(q, st["wq"]), turn(k, st["wk"]), move(v)


def _plain_rope_grad(st):
    case = st["case"]
    cos, sin = _angles(st)

    def back(g):
        if st["perm"] is None:
            return g
        out = torch.empty_like(g)
        out[st["perm"]] = g
        return out

    def turn(g, x, w):
        a, b, rest = _pair_up(back(g), case)
        g = _put_back(a * cos + b * sin, b * cos - a * sin, rest, case)
        if w is None:
            return g, None
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        x = x * r
        dw = (g * x).sum((0, 1))
        g = g * w
        return r * (g - x * (g * x).mean(-1, keepdim=True)), dw

    q, k, _ = _split(st)
    dq, dwq = turn(st["dq"], q, st["wq"])
    dk, dwk = turn(st["dk"], k, st["wk"])
    out = torch.cat((dq, dk, back(st["dv"])), 1).bfloat16()
    return (out, dwq, dwk) if case["norm"] else (out,)


def _plain_attn(st):
    """Rows in chunks (the scores of all rows would not fit), each against its samples' keys."""
    case = st["case"]
    n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
    group, cap, scale = hq // hkv, case["cap"], 1.0 / math.sqrt(d)
    window = case["window"] or n
    q = st["q"].float().view(n, hkv, group, d).permute(1, 2, 0, 3)
    k, v = (st[x].float().transpose(0, 1)[:, None] for x in ("k", "v"))
    train = case["op"] == "attn_train"
    o, lse = torch.empty_like(q), torch.empty((hkv, group, n, 1), device="cuda")
    if train:
        do = st["do"].float().view(n, hkv, group, d).permute(1, 2, 0, 3)
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    index = torch.arange(n, device="cuda")
    rows = max(128, min(2048, (1 << 29) // (hq * n)))
    for a in range(0, n, rows):
        b = min(a + rows, n)
        lo, hi = int(st["first"][a]), int(st["last"][b - 1])
        seg, noise, sample = (st[x] for x in ("seg", "noise", "sample"))
        far = index[a:b, None] - index[None, lo:hi]
        see = (far >= 0) & (far < window)
        see |= (seg[a:b, None] >= 0) & (seg[a:b, None] == seg[None, lo:hi])
        see &= (noise[None, lo:hi] < 0) | (noise[a:b, None] == noise[None, lo:hi])
        see &= sample[a:b, None] == sample[None, lo:hi]
        kk, vv = k[:, :, lo:hi], v[:, :, lo:hi]
        s = q[:, :, a:b] @ kk.transpose(-1, -2) * scale
        if cap:
            t = torch.tanh(s / cap)
            s = cap * t
        if st["slopes"] is not None:
            s = s - st["slopes"].view(hkv, group, 1, 1) * far.abs()
        s = s.masked_fill(~see, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        total = p.sum(-1, keepdim=True)
        lse[:, :, a:b] = m + total.log()
        p = p / total
        o[:, :, a:b] = p @ vv
        if train:
            g = do[:, :, a:b]
            ds = p * (g @ vv.transpose(-1, -2) - (g * o[:, :, a:b]).sum(-1, keepdim=True))
            if cap:
                ds = ds * (1 - t * t)
            dq[:, :, a:b] = ds @ kk * scale
            dk[:, :, lo:hi] += (ds.transpose(-1, -2) @ q[:, :, a:b]).sum(1, keepdim=True) * scale
            dv[:, :, lo:hi] += (p.transpose(-1, -2) @ g).sum(1, keepdim=True)

    def tokens(x):
        return x.permute(2, 0, 1, 3).reshape(n, -1, d).bfloat16()

    out = (tokens(o), lse.view(hq, n))
    return out + (tokens(dq), tokens(dk), tokens(dv)) if train else out


# ----------------------------------------------------------------------------------- exact
def exact(case, seed):
    if case["op"].startswith("rope"):
        return _exact_rope(case, seed)
    heads = case["hq"] * sum(sum(x for _, x in s) ** 2 for s in _spans(case))
    if heads * case["d"] * (14 if case["op"] == "attn_train" else 4) > 6e12:
        return None  # over what 64 bits do in some seconds
    return _exact_attn(case, seed)


def _exact_rope(case, seed):
    """Every pair as a complex number, turned by exp(i position frequency)."""
    st = _inputs(case, seed)
    n, d, rot = case["n"], case["d"], case["rot"]
    freq, axis = _frequencies(case)
    turn = torch.as_tensor(st["pos"].cpu().numpy()[axis].T * freq).cuda()
    turn = torch.polar(torch.ones_like(turn), turn)
    channel = np.arange(rot)
    channel = channel.reshape(2, -1) if case["pairing"] == "halves" else channel.reshape(-1, 2).T
    first, second = (torch.as_tensor(x.copy()).cuda() for x in channel)
    order = torch.arange(n, device="cuda")
    if case["shards"]:
        order = torch.as_tensor(_deal(n, case["shards"])).cuda()

    def rotate(x, by):
        x = x.clone()
        z = torch.complex(x[:, first], x[:, second]) * by
        x[:, first], x[:, second] = z.real, z.imag
        return x

    parts = st["qkv"].split((case["hq"], case["hkv"], case["hkv"]), dim=1)
    out, dws = [], []
    for x, w, g in zip(parts, (st["wq"], st["wk"], None),
                       (st.get("dq"), st.get("dk"), st.get("dv"))):
        dw = torch.zeros(d, dtype=torch.float64, device="cuda")
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for h in range(x.shape[1]):  # a head at a time, for the memory
            xh = x[:, h].double()
            norm = torch.sqrt(xh.pow(2).sum(-1, keepdim=True) / d + EPS)
            moved = len(out) < 2
            if g is None:
                yh = xh if w is None else xh / norm * w.double()
                y[:, h] = (rotate(yh, turn) if moved else yh)[order]
                continue
            gh = torch.empty_like(xh)
            gh[order] = g[:, h].double()
            gh = rotate(gh, turn.conj()) if moved else gh
            if w is not None:
                dw += (gh * xh / norm).sum(0)
                gh = gh * w.double()
                gh = gh / norm - xh * (gh * xh).sum(-1, keepdim=True) / (d * norm ** 3)
            y[:, h] = gh
        out.append(y)
        dws.append(dw)
    if case["op"] == "rope":
        return tuple(out)
    out = torch.cat(out, 1)
    return (out, dws[0], dws[1]) if case["norm"] else (out,)


def _exact_attn(case, seed):
    """Sample by sample and head by head, the gradients by torch's own differentiation."""
    st = _inputs(case, seed)
    hq, hkv, d, n = case["hq"], case["hkv"], case["d"], case["n"]
    train = case["op"] == "attn_train"
    q, k, v = (st[x].double().requires_grad_(train) for x in ("q", "k", "v"))
    o = torch.empty((n, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((hq, n), dtype=torch.float64, device="cuda")
    at = 0
    for s in _spans(case):
        a, at = at, at + sum(x for _, x in s)
        i = torch.arange(a, at, device="cuda")
        seg, noise = st["seg"][a:at], st["noise"][a:at]
        ago = i[:, None] - i
        hidden = ((ago < 0) | (ago >= (case["window"] or n))) & \
            ((seg[:, None] != seg) | (seg < 0))
        hidden |= (noise >= 0) & (noise[:, None] != noise)
        for h in range(hq):
            kh = h // (hq // hkv)
            s = (q[a:at, h] @ k[a:at, kh].T) / d ** 0.5
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            if case["bias"]:
                s = s - float(st["slopes"][h]) * ago.abs()
            s = s.masked_fill(hidden, -math.inf)
            y = torch.softmax(s, -1) @ v[a:at, kh]
            o[a:at, h] = y.detach()
            lse[h, a:at] = torch.logsumexp(s.detach(), -1)
            if train:
                y.backward(st["do"][a:at, h].double())
    return (o, lse, q.grad, k.grad, v.grad) if train else (o, lse)


# ------------------------------------------------------------------------------------ work
def work(case):
    n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":  # q, k and v in and out in 16 bits, the positions
        rows = n * (hq + 2 * hkv) * d
        return {"bytes": 4 * rows + 4 * n * case["axes"], "flops": 6 * rows}
    if case["op"] == "rope_grad":  # the gradients in 32 bits in, in 16 out; q and k for the norm
        rows, normed = n * (hq + 2 * hkv) * d, n * (hq + hkv) * d if case["norm"] else 0
        return {"bytes": 6 * rows + 2 * normed + 4 * n * case["axes"],
                "flops": 6 * rows + 10 * normed}
    token = 2 * n * (2 * hq + 2 * hkv) * d + 4 * n * hq + 12 * n
    if case["op"] == "attn":  # two products over the pairs; q, k, v in, o and lse out
        return {"bytes": token, "flops": 4 * d * hq * _pairs(case)}
    # seven products; the gradient of o in, those of q, k and v out
    return {"bytes": token + 2 * n * (2 * hq + 2 * hkv) * d, "flops": 14 * d * hq * _pairs(case)}
