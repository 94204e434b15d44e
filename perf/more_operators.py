"""What is measured of the operators that build, share and read a paged key-value cache around the
int4 linears: the tables of a serving step made on the GPU, attention of a batch whose sequences
share long prefixes, and cross attention to an encoder's states.

Every case runs in one of two forms on the same inputs: elementary torch operations (`own` false) or
the library's kernels (`own` true)."""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------
# cases


def _tables(name, B, held, nq, every, ends, page, spare=1.0):
    """B sequences that hold up to `held` keys; every `every`-th gets up to nq new tokens, the others
    one; every `ends`-th sequence has come to its end (0: none). spare: the share of the pages needed
    that the ring of free pages holds."""
    c = dict(op="tables", B=B, held=held, nq=nq, every=every, ends=ends, page=page,
             spare=float(spare))
    return dict(c, name=name) if name else c


def _shared(name, B, prefixes, P, rest, nq, rag, alone, Hq, Hkv, D, page, window=0, sinks=0):
    """B sequences over `prefixes` prefixes of up to P keys, each with up to `rest` keys of its own,
    the nq newest of them this call's tokens. Every alone-th sequence has no prefix, and the slot
    after it holds no sequence (0: neither)."""
    c = dict(op="shared", B=B, prefixes=prefixes, P=P, rest=rest, nq=nq, rag=float(rag), alone=alone,
             Hq=Hq, Hkv=Hkv, D=D, page=page, window=window, sinks=sinks)
    return dict(c, name=name) if name else c


def _cross(name, B, nq, n, rag, Hq, Hkv, D, page):
    """B requests of up to nq rows each (1: one each) over up to n states of an encoder."""
    c = dict(op="cross", B=B, nq=nq, n=n, rag=float(rag), Hq=Hq, Hkv=Hkv, D=D, page=page)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decode step of a serving batch: a token for each, three sequences have ended
        _tables("tables decode step", 48, 8192, 1, 1, 16, 16),
        # a step that mixes decode with chunks of prompts, odd sizes, a ring that runs dry
        _tables("tables mixed step", 333, 5000, 777, 11, 9, 32, 0.9),
        # the prompts of a large offline batch at once, about a million tokens
        _tables("tables prompts", 512, 0, 4096, 1, 0, 64),
        # four samples of one question, 1000 tokens: the 7B-class decoder's 28 and 4 heads of 128
        _shared("shared one question", 4, 1, 1000, 90, 1, 0.3, 0, 28, 4, 128, 64),
        # a chat service: one system prompt of 2048, conversations of up to 600 tokens
        _shared("shared system prompt", 64, 1, 2048, 600, 1, 0.9, 0, 28, 4, 128, 16),
        # several tenants with prompts of their own, ragged, some requests without, idle slots
        _shared("shared five prompts", 100, 5, 8000, 1500, 1, 0.6, 10, 28, 4, 128, 64),
        # many questions about one long document
        _shared("shared document", 256, 1, 32768, 200, 1, 0.5, 0, 28, 4, 128, 64),
        # four drafted tokens and one more to verify, for each of 24 sequences, wide heads
        _shared("shared drafts", 24, 2, 2900, 700, 5, 0.5, 0, 16, 4, 256, 32),
        # the newest token of each request over the states of up to 1500 frames, 20 heads of 64
        _cross("cross one token", 12, 1, 1500, 0.5, 20, 20, 64, 64),
        # five beams of each request
        _cross("cross beams", 16, 5, 1500, 0.5, 20, 20, 64, 16),
        # teacher-forced rows over the same states
        _cross("cross rows", 8, 448, 1500, 0.3, 20, 20, 64, 64),
        # a long document's states, shared key-value heads of 128
        _cross("cross long", 2, 2000, 6000, 0.2, 28, 4, 128, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _heads(rng):
    Hkv = rng.choice([1, 2, 4, 8])
    return Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv, rng.choice([64, 80, 128, 128, 256])


def draw(rng):
    op = rng.choice(["tables", "shared", "shared", "shared", "cross", "cross"])
    Hq, Hkv, D = _heads(rng)
    page = rng.choice([16, 32, 64, 128])
    if op == "tables":
        B, nq, every = _log(rng, 1, 1024), _log(rng, 1, 8192), rng.choice([1, 1, 2, 7, 30])
        nq = min(nq, max(1, 1_000_000 * every // B))
        held = rng.choice([0, _log(rng, 1, min(32768, 16_000_000 // B))])
        return _tables(None, B, held, nq, every, rng.choice([0, 0, 3, 20]), page,
                       rng.choice([1.0, 1.0, 0.7]))
    if op == "shared":
        nq = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 200)])
        P = min(_log(rng, 16, 65536), 30_000_000 // (Hkv * D))
        # no larger than the largest listed ones: (row, key) pairs, rows, and keys
        most = min(25_000_000_000 // (P * Hq * D), 12_000_000 // (Hq * D))
        nq = max(1, min(nq, most))
        B = max(1, min(_log(rng, 1, 512), most // nq))
        rest = max(nq, _log(rng, 1, max(1, min(4096, P * 8, 30_000_000 // (B * Hkv * D)))))
        prefixes = min(rng.choice([1, 1, 2, _log(rng, 3, 20)]), B,
                       max(1, 30_000_000 // (P * Hkv * D)))
        window = rng.choice([0, 0, 0, _log(rng, 64, 4096)])
        return _shared(None, B, prefixes, P, rest, nq, rng.choice([0.0, rng.random()]),
                       rng.choice([0, 0, 5]), Hq, Hkv, D, page, window,
                       rng.choice([0, 4, rng.randint(1, 80)]) if window else 0)
    most = 140_000_000_000 // (2 * Hq * D)  # (row, state) pairs, below the largest listed case's
    nq = rng.choice([1, rng.randint(2, 10), _log(rng, 11, 4096)])
    n = min(_log(rng, 1, 16384), most // nq)
    B = max(1, min(_log(rng, 1, 128), most // (nq * n), 30_000_000 // (n * Hkv * D),
                   20_000_000 // (nq * Hq * D)))
    return _cross(None, B, nq, n, rng.choice([0.0, 0.7 * rng.random()]), Hq, Hkv, D, page)


# ---------------------------------------------------------------------------------------------
# inputs


def _spread(most, B, rag, least=1):
    """B lengths up to `most`, the first the longest, lowered by up to the share rag."""
    return [max(least, round(most * (1.0 - rag * ((b * 0.6180339887) % 1.0)))) for b in range(B)]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(
        torch.bfloat16)


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def _pages(c, g, counts, spare=3):
    """Tables of pages in random order, one for each count of pages, and how many pages there are."""
    total = sum(counts) + spare
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(counts), max(max(counts), 1)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for row, n in zip(table, counts):
        row[:n] = order[at:at + n]
        at += n
    return table, total


def _store(c, g, total):
    kv = []
    for _ in range(2):
        t = torch.empty((total, c["page"], c["Hkv"], c["D"]), dtype=torch.bfloat16, device=DEV)
        kv.append(t.normal_(generator=g))
    return kv


def _step(c):
    """(keys held, new tokens, -1 at its end) of each sequence of a tables case."""
    B = c["B"]
    held = [0] * B if c["held"] == 0 else _spread(c["held"], B, 0.9)
    new = _spread(c["nq"], B, 0.8)
    new = [n if b % c["every"] == 0 else 1 for b, n in enumerate(new)]
    if c["ends"]:
        new = [-1 if b % c["ends"] == c["ends"] - 1 else n for b, n in enumerate(new)]
    return held, new


def _needs(c):
    """Pages that each sequence of a tables case holds, and those it will hold."""
    held, new = _step(c)
    have = [-(-n // c["page"]) for n in held]
    return have, [-(-(n + m) // c["page"]) if m >= 0 else h for n, m, h in zip(held, new, have)]


def _groups(c):
    """Of a shared case: each prefix's length, each sequence's prefix (-1: none), its keys and its
    new tokens."""
    P = _spread(c["P"], c["prefixes"], c["rag"])
    rest = _spread(c["rest"], c["B"], c["rag"], c["nq"])
    of, lens, new = [], [], []
    for b, n in enumerate(rest):
        kind = b % c["alone"] if c["alone"] else -1
        g = -1 if kind >= 0 and kind >= c["alone"] - 2 else b * 7 % c["prefixes"]
        idle = kind >= 0 and kind == c["alone"] - 1
        of.append(g)
        lens.append(0 if idle else n + (P[g] if g >= 0 else 0))
        new.append(0 if idle and c["nq"] > 1 else c["nq"])
    return P, of, lens, new


def _rows_of(c):
    """(rows, states) of each request of a cross case."""
    n = _spread(c["n"], c["B"], c["rag"])
    return ([1] * c["B"] if c["nq"] == 1 else _spread(c["nq"], c["B"], c["rag"])), n


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "tables":
        held, new = _step(c)
        have, want = _needs(c)
        fresh = sum(want) - sum(have)
        spare = max(1, int(fresh * c["spare"])) if c["spare"] < 1 else fresh + 7
        table, total = _pages(c, g, [max(a, b) for a, b in zip(have, want)], spare + 1)
        # the first pages of each row are held, the others free
        at = torch.arange(table.shape[1], device=DEV)
        table = torch.where(at < _ints(have)[:, None], table, -1)
        mark = torch.zeros(total + 1, dtype=torch.bool, device=DEV)
        mark[table.flatten().long()] = True  # (-1: the place after the last)
        free = torch.nonzero(~mark[:total]).flatten()
        free = free[torch.randperm(free.shape[0], generator=g, device=DEV)][:spare]
        head = int(torch.randint(total, (1,), generator=g, device=DEV))
        ring = torch.full((total,), -1, dtype=torch.int32, device=DEV)
        ring[(head + torch.arange(free.shape[0], device=DEV)) % total] = free.to(torch.int32)
        starts = torch.tensor([0] + [max(n, 0) for n in new]).cumsum(0)
        return dict(case=c, kv_len=_ints(held), n_new=_ints(new), table=table, ring=ring,
                    spans=torch.stack([torch.zeros_like(_ints(have)), _ints(have)], 1).contiguous(),
                    state=_ints([head, free.shape[0], 0]), T=int(starts[-1]) + c["B"] % 3)
    if c["op"] == "shared":
        P, of, lens, new = _groups(c)
        counts = [-(-n // c["page"]) for n in lens]
        table, total = _pages(c, g, counts + [-(-n // c["page"]) for n in P])
        k, v = _store(c, g, total)
        s = dict(case=c, k=k, v=v, table=table[:c["B"]].clone(), prefix_table=table[c["B"]:].clone(),
                 prefix_len=_ints(P), prefix_of=_ints(of), P=P,
                 members=[_ints([b for b, x in enumerate(of) if x == i], torch.int64)
                          for i in range(len(P))])
    else:
        new, lens = _rows_of(c)
        table, total = _pages(c, g, [-(-n // c["page"]) for n in lens])
        k, v = _store(c, g, total)
        s = dict(case=c, k=k, v=v, table=table)
    starts = torch.tensor([0] + new).cumsum(0)
    T = int(starts[-1])
    s.update(kv_len=_ints(lens), q_start=starts.to(torch.int32).to(DEV), T=T,
             q=_randn(g, T, c["Hq"] * c["D"], scale=2.0),  # scores spread over several units
             scale=1.0 / math.sqrt(c["D"]))
    return s


# ---------------------------------------------------------------------------------------------
# the plain forms


def _plain_tables(s):
    page, T, table, ring = s["case"]["page"], s["T"], s["table"], s["ring"]
    B, cols = table.shape
    R = ring.shape[0]
    L, begin, end = s["kv_len"], s["spans"][:, 0], s["spans"][:, 1]
    head, count = s["state"][0], s["state"][1]
    over = s["n_new"] < 0
    m = s["n_new"].clamp(min=0)
    q_start = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    q_start[1:] = m.cumsum(0)
    want = torch.where(over, end, ((L + m + page - 1) // page).clamp(max=cols))
    fresh = (want - end).clamp(min=0)
    first = fresh.cumsum(0) - fresh
    given = torch.minimum((count - first).clamp(min=0), fresh)
    gone = torch.where(over, end - begin, 0)
    # new entries, where the ring still has pages
    at = torch.arange(cols, device=DEV)[None]
    k = first[:, None] + at - end[:, None]
    page_of = torch.where(k < count, ring[(head + k.clamp(min=0)) % R], -1)
    new = (at >= end[:, None]) & (at < want[:, None])
    # pages that come back, behind those of the ring (a place after the last for all others)
    back = (at >= begin[:, None]) & (at < end[:, None]) & over[:, None]
    to = (head + count + (gone.cumsum(0) - gone)[:, None] + at - begin[:, None]) % R
    wide = torch.cat([ring, ring[:1]])
    wide[torch.where(back, to, R).flatten()] = torch.where(back, table, 0).flatten()
    ring.copy_(wide[:R])
    table.copy_(torch.where(new, page_of.to(torch.int32), table))
    rows = torch.arange(T, device=DEV, dtype=torch.int32)
    seq = torch.bucketize(rows, q_start[1:], right=True)
    used = seq < B
    b = seq.clamp(max=B - 1)
    pos = L[b] + rows - q_start[b]
    col = pos // page
    entry = torch.where(col < cols, table[b, col.clamp(max=cols - 1).long()], -1).long()
    slots = torch.where(used & (entry >= 0), entry * page + pos % page, -1)
    taken = given.sum()
    return {"q_start": q_start, "slots": slots,
            "seqs": torch.where(used, seq, -1).to(torch.int32),
            "positions": torch.where(used, pos, -1).to(torch.int32),
            "kv_len": torch.where(over, 0, L + m).to(torch.int32),
            "spans": torch.stack([torch.where(over, 0, begin), torch.where(over, 0, end + given)],
                                 1).to(torch.int32),
            "state": torch.stack([(head + taken) % R, count - taken + gone.sum(),
                                  fresh.sum() - taken]).to(torch.int32),
            "table": table, "ring": ring}


def _padded(s, nq):
    """Rows of q by sequence, [B][nq][Hq][D], and where each one stands (-1: none)."""
    c = s["case"]
    count = s["q_start"][1:] - s["q_start"][:-1]
    at = torch.arange(nq, device=DEV)
    rows = (s["q_start"][:-1, None] + at).clamp_(max=s["T"] - 1).long()
    pos = torch.where(at < count[:, None], (s["kv_len"] - count)[:, None] + at, -1)
    return s["q"][rows].view(c["B"], nq, c["Hq"], c["D"]), pos


def _packed(s, y, nq):
    """[B][nq][...] back to the rows of q."""
    at = torch.arange(s["T"], device=DEV, dtype=torch.int32)
    seq = torch.bucketize(at, s["q_start"][1:], right=True).long()
    return y[seq, (at - s["q_start"][seq]).long()]


def _weigh(p, v):
    """Scores (-inf: hidden) and values -> maximum, sum of weights, weighted sums."""
    m = p.amax(-1, keepdim=True).clamp_min_(-1e30)
    p = (p - m).exp_()
    return m, p.sum(-1, keepdim=True), torch.matmul(p, v)


def _plain_shared(s):
    c = s["case"]
    B, nq, Hq, Hkv, D, page = c["B"], c["nq"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    q, pos = _padded(s, nq)
    q = q.view(B, nq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq, D).float()

    def hide(p, j, pos):  # p [...][G * nq][keys], j and pos up to the heads
        out = j > pos
        if c["window"]:
            out |= (j <= pos - c["window"]) & (j >= c["sinks"])
        shape = p.shape
        return p.view(*shape[:-2], G, nq, shape[-1]).masked_fill_(out, -math.inf).view(shape)

    # the keys of each sequence's own
    P = torch.where(s["prefix_of"] >= 0, s["prefix_len"][s["prefix_of"].clamp(min=0).long()], 0)
    j = P[:, None] + torch.arange(c["rest"], device=DEV)
    at = s["table"].gather(1, (j // page).clamp(max=s["table"].shape[1] - 1).long()).long()
    k = s["k"][at, (j % page).long()].permute(0, 2, 1, 3).float()
    v = s["v"][at, (j % page).long()].permute(0, 2, 1, 3).float()
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    m, l, o = _weigh(hide(p, j[:, None, None, None, :], pos[:, None, None, :, None]), v)
    # each prefix once for its sequences, joined with the above
    for g, b in enumerate(s["members"]):
        if b.shape[0] == 0:
            continue
        j = torch.arange(s["P"][g], device=DEV)
        at = s["prefix_table"][g][j // page].long()
        k = s["k"][at, j % page].permute(1, 0, 2).float()
        v = s["v"][at, j % page].permute(1, 0, 2).float()
        x = q[b].transpose(0, 1).reshape(Hkv, -1, D)
        p = torch.matmul(x, k.transpose(-1, -2)).mul_(s["scale"]).view(Hkv, -1, G * nq, s["P"][g])
        p = hide(p, j, pos[b][None, :, None, :, None]).view(Hkv, -1, s["P"][g])
        m1, l1, o1 = (x.view(Hkv, b.shape[0], G * nq, -1).transpose(0, 1) for x in _weigh(p, v))
        top = torch.maximum(m[b], m1)
        f, f1 = (m[b] - top).exp(), (m1 - top).exp()
        l[b], o[b] = l[b] * f + l1 * f1, o[b] * f + o1 * f1
    y = o / torch.where(l > 0, l, 1.0)
    y = y.view(B, Hkv, G, nq, D).permute(0, 3, 1, 2, 4).reshape(B, nq, Hq * D)
    return _packed(s, y, nq).to(torch.bfloat16)


def _plain_cross(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    nq, G = c["nq"], Hq // Hkv
    q, _ = _padded(s, nq)
    q = q.view(B, nq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq, D).float()
    at = s["table"].clamp(min=0).long()
    n = at.shape[1] * c["page"]
    k = s["k"][at].view(B, n, Hkv, D).permute(0, 2, 1, 3).float()
    v = s["v"][at].view(B, n, Hkv, D).permute(0, 2, 1, 3).float()
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    hidden = torch.arange(n, device=DEV) >= s["kv_len"][:, None]
    _, l, o = _weigh(p.masked_fill_(hidden[:, None, None], -math.inf), v)
    y = o / torch.where(l > 0, l, 1.0)
    y = y.view(B, Hkv, G, nq, D).permute(0, 3, 1, 2, 4).reshape(B, nq, Hq * D)
    return _packed(s, y, nq).to(torch.bfloat16)


PLAIN = {"tables": _plain_tables, "shared": _plain_shared, "cross": _plain_cross}


# ---------------------------------------------------------------------------------------------
# the library


def _own(s):
    import int4_weight_only_amd as w4

    c = s["case"]
    if c["op"] == "tables":
        q_start, slots, seqs, positions, kv_len, spans, state = w4.w4_batch_tables(
            s["kv_len"], s["n_new"], s["spans"], s["table"], c["page"], s["ring"], s["state"],
            s["T"])
        return {"q_start": q_start, "slots": slots, "seqs": seqs, "positions": positions,
                "kv_len": kv_len, "spans": spans, "state": state, "table": s["table"],
                "ring": s["ring"]}
    if c["op"] == "shared":
        return w4.w4_attn_shared(
            s["q"], s["k"], s["v"], s["table"], s["kv_len"], s["prefix_of"], s["prefix_table"],
            s["prefix_len"], q_start=s["q_start"] if c["nq"] > 1 else None, scale=s["scale"],
            window=c["window"], sinks=c["sinks"])
    return w4.w4_attn_cross(s["q"], s["k"], s["v"], s["table"], s["kv_len"],
                            q_start=s["q_start"] if c["nq"] > 1 else None, scale=s["scale"])


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without


def _seen(c, m, n, lo, hi):
    """Of m tokens, the newest of n keys: how many pairs with the keys lo .. hi - 1 they see, and how
    many of those keys any of them sees."""
    W, S = c["window"], c["sinks"]
    pairs, keys, upto = 0, 0, lo
    for p in range(max(n - m, 0), n):
        end = min(p + 1, hi)
        start = max(lo, p + 1 - W) if W else lo
        early = max(min(S, start, end) - lo, 0) if W else 0
        pairs += max(end - start, 0) + early
        keys += max(end - max(start, upto), 0) + (early if p == max(n - m, 0) else 0)
        upto = max(upto, end)
    return pairs, keys


def work(case):
    c = case
    if c["op"] == "tables":
        held, new = _step(c)
        have, want = _needs(c)
        back = sum(h for h, n in zip(have, new) if n < 0)
        T = sum(max(n, 0) for n in new) + c["B"] % 3
        return {"bytes": 16 * T + 36 * c["B"] + 8 * (sum(want) - sum(have) + back), "flops": 0}
    if c["op"] == "shared":
        P, of, lens, new = _groups(c)
        pairs = keys = 0
        seen = [0] * len(P)
        for g, n, m in zip(of, lens, new):
            m = min(m, n)
            cut = P[g] if g >= 0 else 0
            a, b = _seen(c, m, n, cut, n)
            pairs, keys = pairs + a, keys + b
            if g >= 0:
                a, b = _seen(c, m, n, 0, cut)
                pairs, seen[g] = pairs + a, max(seen[g], b)
        keys += sum(seen)
        T = sum(new)
    else:
        new, lens = _rows_of(c)
        pairs, keys, T = sum(m * n for m, n in zip(new, lens)), sum(lens), sum(new)
    return {"bytes": keys * c["Hkv"] * c["D"] * 4 + T * c["Hq"] * c["D"] * 4,
            "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---------------------------------------------------------------------------------------------
# the definitions, one sequence after the other, in 64 bits


def _exact_tables(s):
    page, T = s["case"]["page"], s["T"]
    table, ring, spans, kv_len = (s[x].cpu().numpy().copy()
                                  for x in ("table", "ring", "spans", "kv_len"))
    head, count, _ = s["state"].tolist()
    R, cols = ring.shape[0], table.shape[1]
    took = back = missing = 0
    starts, slots, seqs, positions = [0], [], [], []
    for b, m in enumerate(s["n_new"].tolist()):
        begin, end = spans[b]
        if m < 0:
            for p in table[b, begin:end]:
                ring[(head + count + back) % R] = p
                back += 1
            spans[b], kv_len[b] = 0, 0
            starts.append(starts[-1])
            continue
        n = int(kv_len[b])
        for col in range(end, min(-(-(n + m) // page), cols)):
            if took < count:
                table[b, col] = ring[(head + took) % R]
                took += 1
                spans[b, 1] = col + 1
            else:
                table[b, col] = -1
                missing += 1
        for p in range(n, n + m):
            e = int(table[b, p // page]) if p // page < cols else -1
            slots.append(e * page + p % page if e >= 0 else -1)
            positions.append(p)
        seqs += [b] * m
        kv_len[b] = n + m
        starts.append(starts[-1] + m)
    pad = [-1] * (T - starts[-1])
    out = {"q_start": starts, "slots": slots + pad, "seqs": seqs + pad,
           "positions": positions + pad, "kv_len": kv_len, "spans": spans,
           "state": [(head + took) % R, count - took + back, missing], "table": table, "ring": ring}
    return {k: torch.as_tensor(x, dtype=torch.float64) for k, x in out.items()}


def _exact_attention(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    y = torch.zeros(s["T"], Hkv, Hq // Hkv, D, dtype=torch.float64, device=DEV)
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    of = s["prefix_of"].tolist() if c["op"] == "shared" else [-1] * c["B"]
    for b, n in enumerate(lens):
        m = starts[b + 1] - starts[b]
        if n == 0 or m == 0:
            continue
        j = torch.arange(n, device=DEV)
        pages = s["table"][b][j // page].long()
        if of[b] >= 0:
            cut = min(s["P"][of[b]], n)
            pages[:cut] = s["prefix_table"][of[b]][j[:cut] // page].long()
        seen = torch.ones(m, n, dtype=torch.bool, device=DEV)
        if c["op"] == "shared":
            i = torch.arange(n - m, n, device=DEV)[:, None]
            seen = j <= i
            if c["window"]:
                seen &= (j > i - c["window"]) | (j < c["sinks"])
        q = s["q"][starts[b]:starts[b + 1]].double().view(m, Hkv, Hq // Hkv, D)
        for h in range(Hkv):
            k, v = s["k"][pages, j % page, h].double(), s["v"][pages, j % page, h].double()
            for i in range(Hq // Hkv):
                a = torch.where(seen, s["scale"] * (q[:, h, i] @ k.T), -math.inf)
                y[starts[b]:starts[b + 1], h, i] = torch.softmax(a, 1) @ v
    return y.view(s["T"], Hq * D)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_tables(s) if case["op"] == "tables" else _exact_attention(s)
