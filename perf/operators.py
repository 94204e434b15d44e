"""What is measured of the decoder operators around the int4 linears: rotary positions with the
cache append, attention of one new token and of whole prompts over a paged key-value cache (with an
optional sliding window and sink tokens), and the residual norm.

Every case runs in one of two forms on the same inputs: elementary torch operations in 32 bits
(`own` false) or the library's kernels (`own` true)."""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------
# cases


def _rope(name, B, nq, prior, Hq, Hkv, D, rot, layout, page, theta=1e6, scaled=1.0):
    """B sequences of up to nq new tokens each, after up to `prior` cached ones; `scaled`: the
    factor the context is stretched by (frequencies divided, amplitude raised)."""
    c = dict(op="rope", B=B, nq=nq, prior=prior, Hq=Hq, Hkv=Hkv, D=D, rot=rot, layout=layout,
             page=page, theta=float(theta), scaled=float(scaled))
    return dict(c, name=name) if name else c


def _norm(name, T, d, f32_residual, post, gate, alpha):
    """T tokens of width d; residual stream in fp32 or bf16; a norm of the block's output or none;
    gate "none", "channel" (one vector) or "token" (a row each)."""
    c = dict(op="norm", T=T, d=d, f32_residual=f32_residual, post=post, gate=gate,
             alpha=float(alpha))
    return dict(c, name=name) if name else c


def _decode(name, B, n, rag, idle, Hq, Hkv, D, page, window, sinks):
    """B sequences with up to n keys each (rag: the share by which lengths vary; idle: every
    idle-th slot of the batch holds no sequence)."""
    c = dict(op="decode", B=B, n=n, rag=float(rag), idle=idle, Hq=Hq, Hkv=Hkv, D=D, page=page,
             window=window, sinks=sinks)
    return dict(c, name=name) if name else c


def _prefill(name, B, nq, prior, rag, Hq, Hkv, D, page, window, sinks):
    """B sequences of up to nq new tokens each after up to `prior` cached ones."""
    c = dict(op="prefill", B=B, nq=nq, prior=prior, rag=float(rag), Hq=Hq, Hkv=Hkv, D=D,
             page=page, window=window, sinks=sinks)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decode step of one user: the 7B-class decoder's 28 query and 4 key-value heads of 128
        _rope("rope one token", 1, 1, 4096, 28, 4, 128, 128, "half", 64),
        # prompts of the same decoder, about 13000 tokens in a batch of eight
        _rope("rope prompts", 8, 2048, 0, 28, 4, 128, 128, "half", 64),
        # a chunk of a long document: adjacent pairs, half of the head rotated, context x 4
        _rope("rope long chunk", 2, 1000, 100000, 16, 8, 80, 40, "interleaved", 16, 1e4, 4.0),
        # the norm between two blocks of a decode step, hidden size 3584
        _norm("norm one token", 1, 3584, False, False, "none", 1.0),
        # the same over a prefill batch, norms on both sides, a gated branch, fp32 residual stream
        _norm("norm prompts", 8192, 3584, True, True, "channel", 0.7),
        # one user's decode step after a 4097-token conversation
        _decode("decode one sequence", 1, 4097, 0.0, 0, 28, 4, 128, 64, 0, 0),
        # a serving batch: ragged lengths, two idle slots
        _decode("decode batch", 32, 8192, 0.9, 16, 28, 4, 128, 16, 0, 0),
        # few users with very long contexts
        _decode("decode long", 4, 131072, 0.1, 0, 28, 4, 128, 64, 0, 0),
        # a sliding-window layer: 1024 recent keys and 4 sinks, wide heads
        _decode("decode window", 32, 8192, 0.5, 0, 16, 4, 256, 32, 1024, 4),
        # a short question
        _prefill("prefill short", 1, 77, 0, 0.0, 28, 4, 128, 64, 0, 0),
        # prompts of up to 4096 tokens
        _prefill("prefill prompts", 3, 4096, 0, 0.4, 28, 4, 128, 64, 0, 0),
        # a chunk of a long prompt in a sliding-window layer with sinks, wide heads
        _prefill("prefill window", 2, 4096, 4096, 0.1, 16, 4, 256, 32, 1024, 4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    Hkv = rng.choice([1, 2, 4, 8])
    return Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv, rng.choice([64, 80, 128, 128, 256])


def draw(rng):
    op = rng.choice(["rope", "norm", "decode", "decode", "prefill", "prefill"])
    Hq, Hkv, D = _heads(rng)
    page = rng.choice([16, 32, 64, 128])
    window = rng.choice([0, 0, _log(rng, 64, 4096)])
    sinks = rng.choice([0, 4, rng.randint(1, 80)]) if window else 0
    if op == "rope":
        nq = min(_log(rng, 1, 4096), 40_000_000 // (Hq * D))
        B = _log(rng, 1, min(64, 40_000_000 // (nq * Hq * D)))
        rot = rng.choice([D, D // 2])
        return _rope(None, B, nq, rng.choice([0, _log(rng, 1, 100000 // B)]), Hq, Hkv, D, rot,
                     rng.choice(["half", "interleaved"]), page, rng.choice([1e4, 1e6]),
                     rng.choice([1.0, 4.0]))
    if op == "norm":
        d = rng.choice([_log(rng, 64, 16384), 8 * _log(rng, 8, 2048)])
        return _norm(None, _log(rng, 1, min(16384, 29_000_000 // d)), d, rng.random() < 0.5,
                     rng.random() < 0.5, rng.choice(["none", "channel", "token"]),
                     rng.uniform(0.1, 1.5))
    if op == "decode":
        n = _log(rng, 1, 131072)
        B = _log(rng, 1, max(1, min(128, 200_000_000 // (n * Hkv * D))))
        return _decode(None, B, n, rng.choice([0.0, rng.random()]), rng.choice([0, 0, 5]), Hq,
                       Hkv, D, page, window, sinks)
    most = 70_000_000_000 // (Hq * D)  # (token, key) pairs, no more than the largest listed case
    nq = min(_log(rng, 1, 4096), math.isqrt(most))
    prior = rng.choice([0, min(_log(rng, 1, 16384), most // nq - nq)])
    B = _log(rng, 1, min(16, most // (nq * (nq + prior))))
    return _prefill(None, B, nq, prior, rng.choice([0.0, 0.7 * rng.random()]), Hq, Hkv, D, page,
                    window, sinks)


# ---------------------------------------------------------------------------------------------
# inputs


def _spread(most, B, rag, idle=0):
    """B lengths up to `most`, the first the longest, lowered by up to the share rag."""
    got = [max(1, round(most * (1.0 - rag * ((b * 0.6180339887) % 1.0)))) for b in range(B)]
    return [0 if idle and b % idle == idle - 1 else x for b, x in enumerate(got)]


def _lengths(c):
    """(new tokens, keys after them) of each sequence, a function of the case alone."""
    if c["op"] == "decode":
        n = _spread(c["n"], c["B"], c["rag"], c["idle"])
        return [1] * c["B"], n
    rag = c.get("rag", 0.5)
    nq = _spread(c["nq"], c["B"], rag)
    prior = _spread(c["prior"], c["B"], rag) if c["prior"] else [0] * c["B"]
    return nq, [a + b for a, b in zip(nq, prior)]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)


def _cache(c, g, lens):
    """A paged cache with its pages in random order, a few of them free, and filled slots."""
    pages = [-(-n // c["page"]) for n in lens]
    cols = max(max(pages), 1)
    total = sum(pages) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    shape = (total, c["page"], c["Hkv"], c["D"])
    kv = []
    for _ in range(2):
        t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        t.normal_(generator=g)
        kv.append(t)
    return kv[0], kv[1], table.to(DEV)


def _inv_freq(c):
    half = c["rot"] // 2
    i = torch.arange(half, dtype=torch.float64)
    return ((c["theta"] ** (-2.0 * i / c["rot"])) / c["scaled"]).to(torch.float32).to(DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        ld = (d + 7) // 8 * 8  # rows of a wider buffer where the width is odd
        s = dict(case=c, x=_randn(g, T, ld)[:, :d],
                 residual=_randn(g, T, ld, scale=3.0, dtype=torch.float32 if c["f32_residual"]
                                 else torch.bfloat16)[:, :d],
                 w_pre=_randn(g, d, scale=0.2) + 1.0,
                 w_post=_randn(g, d, scale=0.2) + 1.0 if c["post"] else None, gate=None)
        if c["gate"] == "channel":
            s["gate"] = torch.sigmoid(_randn(g, d))
        elif c["gate"] == "token":
            s["gate"] = torch.sigmoid(_randn(g, T, ld))[:, :d]
        return s
    nq, lens = _lengths(c)
    k, v, table = _cache(c, g, lens)
    starts = [0]
    for x in nq:
        starts.append(starts[-1] + x)
    T = starts[-1]
    s = dict(case=c, k=k, v=v, table=table, nq=max(nq), T=T,
             kv_len=torch.tensor(lens, dtype=torch.int32, device=DEV),
             q_start=torch.tensor(starts, dtype=torch.int32, device=DEV))
    if c["op"] == "rope":
        s["qkv"] = _randn(g, T, (c["Hq"] + 2 * c["Hkv"]) * c["D"])
        s["inv_freq"] = _inv_freq(c)
        s["factor"] = 0.1 * math.log(c["scaled"]) + 1.0
    else:
        s["q"] = _randn(g, T, c["Hq"] * c["D"], scale=2.0)  # scores spread over several units
        s["scale"] = 1.0 / math.sqrt(c["D"])
    return s


# ---------------------------------------------------------------------------------------------
# the plain forms


def _rows(s):
    """The sequence of each token row, and its place among that sequence's new tokens."""
    at = torch.arange(s["T"], device=DEV, dtype=torch.int32)
    seq = torch.bucketize(at, s["q_start"][1:], right=True)
    return seq, at - s["q_start"][seq]


def _plain_rope(s):
    c = s["case"]
    Hq, Hkv, D, R, page = c["Hq"], c["Hkv"], c["D"], c["rot"], c["page"]
    seq, i = _rows(s)
    pos = s["kv_len"][seq] - (s["q_start"][seq + 1] - s["q_start"][seq]) + i
    x = s["qkv"].float().view(s["T"], Hq + 2 * Hkv, D)
    ang = pos.float()[:, None] * s["inv_freq"][None]
    cos, sin = (ang.cos() * s["factor"])[:, None], (ang.sin() * s["factor"])[:, None]
    qk, r = x[:, :Hq + Hkv], x[:, :Hq + Hkv, :R]
    if c["layout"] == "half":
        a, b = r[..., :R // 2], r[..., R // 2:]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    out = torch.cat([r, qk[..., R:]], -1).to(torch.bfloat16)
    where = s["table"][seq, (pos // page).long()].long()
    slot = (pos % page).long()
    s["k"][where, slot] = out[:, Hq:]
    s["v"][where, slot] = s["qkv"].view(s["T"], Hq + 2 * Hkv, D)[:, Hq + Hkv:]
    return {"q": out[:, :Hq].reshape(s["T"], Hq * D), "k": s["k"], "v": s["v"]}


def _rms(u, w):
    return u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-6) * w.float()


def _plain_norm(s):
    n = s["x"].float()
    if s["w_post"] is not None:
        n = _rms(n, s["w_post"])
    if s["gate"] is not None:
        n = n * s["gate"].float()
    r = s["residual"].float() + s["case"]["alpha"] * n
    return {"y": _rms(r, s["w_pre"]).to(torch.bfloat16), "residual": r.to(s["residual"].dtype)}


def _plain_attention(s, q, pos):
    """q [B][nq][Hq][D], pos [B][nq] (below 0: a row of padding) -> [B][nq][Hq * D]."""
    c = s["case"]
    B, nq, Hq, D = q.shape
    Hkv, G = c["Hkv"], c["Hq"] // c["Hkv"]
    at = s["table"].long()
    L = at.shape[1] * c["page"]
    k = s["k"][at].view(B, L, Hkv, D).permute(0, 2, 1, 3).float()
    v = s["v"][at].view(B, L, Hkv, D).permute(0, 2, 1, 3).float()
    q = q.view(B, nq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq, D).float()
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, G, nq, L)
    j = torch.arange(L, device=DEV)
    hidden = j > pos[..., None]
    if c["window"]:
        hidden |= (j <= pos[..., None] - c["window"]) & (j >= c["sinks"])
    p.masked_fill_(hidden[:, None, None], -math.inf)
    p -= p.amax(-1, keepdim=True).clamp_min_(-1e30)
    p.exp_()
    total = p.sum(-1, keepdim=True).view(B, Hkv, G * nq, 1)
    y = torch.matmul(p.view(B, Hkv, G * nq, L), v) / torch.where(total > 0, total, 1.0)
    return y.view(B, Hkv, G, nq, D).permute(0, 3, 1, 2, 4).reshape(B, nq, Hq * D)


def _plain_decode(s):
    c = s["case"]
    q = s["q"].view(c["B"], 1, c["Hq"], c["D"])
    return _plain_attention(s, q, s["kv_len"][:, None] - 1)[:, 0].to(torch.bfloat16)


def _plain_prefill(s):
    c = s["case"]
    seq, i = _rows(s)
    count = s["q_start"][1:] - s["q_start"][:-1]
    slot = torch.arange(s["nq"], device=DEV)
    rows = (s["q_start"][:-1, None] + slot).clamp_(max=s["T"] - 1).long()
    pos = torch.where(slot < count[:, None], (s["kv_len"] - count)[:, None] + slot, -1)
    y = _plain_attention(s, s["q"][rows].view(c["B"], s["nq"], c["Hq"], c["D"]), pos)
    return y[seq.long(), i.long()].to(torch.bfloat16)


PLAIN = {"rope": _plain_rope, "norm": _plain_norm, "decode": _plain_decode,
         "prefill": _plain_prefill}


# ---------------------------------------------------------------------------------------------
# the library


def _own(s):
    import int4_weight_only_amd as w4

    c = s["case"]
    if c["op"] == "rope":
        q = w4.w4_rope_append(
            s["qkv"], c["Hq"], s["k"], s["v"], s["table"], s["kv_len"], s["inv_freq"],
            q_start=s["q_start"], factor=s["factor"],
            layout=w4.W4_ROPE_HALF if c["layout"] == "half" else w4.W4_ROPE_INTERLEAVED)
        return {"q": q, "k": s["k"], "v": s["v"]}
    if c["op"] == "norm":
        y, r = w4.w4_residual_norm(s["x"], s["residual"], s["w_pre"], w_post=s["w_post"],
                                   gate=s["gate"], alpha=c["alpha"], eps=1e-6)
        return {"y": y, "residual": r}
    if c["op"] == "decode":
        return w4.w4_attn_decode(s["q"], s["k"], s["v"], s["table"], s["kv_len"],
                                 scale=s["scale"], window=c["window"], sinks=c["sinks"])
    return w4.w4_attn_prefill(s["q"], s["k"], s["v"], s["table"], s["kv_len"], s["q_start"],
                              scale=s["scale"], window=c["window"], sinks=c["sinks"])


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without


def _visible(c):
    """Visible (token, key) pairs, and keys that some token of their sequence sees."""
    pairs = keys = 0
    W, S = c["window"], c["sinks"]
    for m, n in zip(*_lengths(c)):
        m = min(m, n)
        if not W:
            pairs += m * n - m * (m - 1) // 2
            keys += n
            continue
        seen = [min(n - m + i + 1, W) + min(S, max(n - m + i + 1 - W, 0)) for i in range(m)]
        pairs += sum(seen)
        keys += min(n, W + m - 1 + S) if m else 0
    return pairs, keys


def work(case):
    c = case
    if c["op"] == "norm":
        a = c["T"] * c["d"]
        rows = a * (2 + (4 if c["f32_residual"] else 2) * 2 + 2)
        return {"bytes": rows + c["d"] * 2 * (1 + c["post"] + (c["gate"] == "channel"))
                + (2 * a if c["gate"] == "token" else 0), "flops": 10 * a}
    if c["op"] == "rope":
        T = sum(_lengths(c)[0])
        width = (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": T * width * 4 + c["rot"] * 2,
                "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    pairs, keys = _visible(c)
    T = sum(_lengths(c)[0])
    return {"bytes": keys * c["Hkv"] * c["D"] * 4 + T * c["Hq"] * c["D"] * 4,
            "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_rope(s):
    c = s["case"]
    Hq, Hkv, D, R = c["Hq"], c["Hkv"], c["D"], c["rot"]
    k, v = s["k"].double(), s["v"].double()
    q = torch.empty(s["T"], Hq, D, dtype=torch.float64, device=DEV)
    nq, lens = _lengths(c)
    row = 0
    first = [p for p in range(R // 2)] if c["layout"] == "half" else list(range(0, R, 2))
    second = [p + (R // 2 if c["layout"] == "half" else 1) for p in first]
    for b, (m, n) in enumerate(zip(nq, lens)):
        x = s["qkv"][row:row + m].double().view(m, Hq + 2 * Hkv, D)
        pos = torch.arange(n - m, n, device=DEV)
        turn = torch.polar(torch.full((m, R // 2), s["factor"], dtype=torch.float64, device=DEV),
                           pos.double()[:, None] * s["inv_freq"].double())[:, None]
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        q[row:row + m] = y[:, :Hq]
        page = s["table"][b][pos // c["page"]].long()
        k[page, pos % c["page"]] = y[:, Hq:Hq + Hkv]
        v[page, pos % c["page"]] = x[:, Hq + Hkv:]
        row += m
    return {"q": q.view(s["T"], Hq * D), "k": k, "v": v}


def _exact_norm(s):
    def scaled(u, w):
        return u * w.double() / (u.square().sum(1, keepdim=True) / u.shape[1] + 1e-6).sqrt()

    n = s["x"].double()
    n = scaled(n, s["w_post"]) if s["w_post"] is not None else n
    n = n * (s["gate"].double() if s["gate"] is not None else 1.0)
    r = s["residual"].double() + s["case"]["alpha"] * n
    return {"y": scaled(r, s["w_pre"]), "residual": r}


def _exact_attention(s):
    """One sequence and one key-value head at a time, one query head's score matrix in memory."""
    c = s["case"]
    D, G = c["D"], c["Hq"] // c["Hkv"]
    nq, lens = _lengths(c)
    y = torch.zeros(s["T"], c["Hq"], D, dtype=torch.float64, device=DEV)
    row = 0
    for b, (m, n) in enumerate(zip(nq, lens)):
        if n:
            j = torch.arange(n, device=DEV)
            page = s["table"][b][j // c["page"]].long()
            i = torch.arange(n - m, n, device=DEV)[:, None]
            seen = j[None] <= i
            if c["window"]:
                seen &= (j[None] > i - c["window"]) | (j[None] < c["sinks"])
            for h in range(c["Hkv"]):
                k = s["k"][page, j % c["page"], h].double()
                v = s["v"][page, j % c["page"], h].double()
                for h2 in range(h * G, h * G + G):
                    q = s["q"][row:row + m].view(m, c["Hq"], D)[:, h2].double()
                    a = torch.where(seen, s["scale"] * (q @ k.T), -math.inf)
                    y[row:row + m, h2] = torch.softmax(a, 1) @ v
        row += m
    return y.view(s["T"], c["Hq"] * D)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rope", "norm"):
        return _exact_rope(s) if op == "rope" else _exact_norm(s)
    if work(case)["flops"] > 2e12:
        return None
    return _exact_attention(s)
