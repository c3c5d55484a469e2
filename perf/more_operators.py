"""What a chunk of new tokens needs around the GEMVs, as cases that can be timed and compared.

A chunk is a piece of a prompt, the draft tokens of a speculative step, or both beside sequences
that decode one token each.  Its rows come as one ragged batch: rows starts[i] .. starts[i + 1] - 1
are the last tokens of sequence seqs[i].  Three operators, each in a plain form (elementary torch
operations in fp32, rounded once) and as the calls a program makes of the library:

  append  queries and keys normalised for each head (optional), rotated by their positions, keys and
          values put into their pages, queries into a tensor for the attention
  chunk   causal attention of the new tokens over the paged cache, with capped scores, a sliding
          window or a bias by distance where a case has them
  grow    pages for the new tokens: ended sequences released, their slots grown by new prompts

`own` selects the side: False the plain form, True the library.
"""
import math
import random

import torch

own = False

ACT = {"f16": torch.float16, "bf16": torch.bfloat16}
BASE = 500000.0  # of the rotation's frequencies


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one user's next token: the normalised, rotated heads of one layer; latency counts
        {"name": "append_1", "lot": 1, "op": "append", "act": "bf16", "n": 1, "big": 1, "new": 1,
         "ragged": False, "past": 1000, "idle": 0, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "inter": False, "norm": True, "stretch": 1, "ps": 16, "layout": "head"},
        # pieces of several prompts beside decoding sequences, padded entries, half of each head
        # rotated in pairs, token-major pages
        {"name": "append_odd", "lot": 2, "op": "append", "act": "f16", "n": 37, "big": 6, "new": 131,
         "ragged": True, "past": 2100, "idle": 3, "Hq": 24, "Hkv": 8, "D": 64, "rot": 32,
         "inter": True, "norm": False, "stretch": 1, "ps": 32, "layout": "token"},
        # a long prompt's large piece, far positions on frequencies stretched for them
        {"name": "append_8192", "lot": 3, "op": "append", "act": "bf16", "n": 1, "big": 1, "new": 8192,
         "ragged": False, "past": 24000, "idle": 0, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "inter": False, "norm": True, "stretch": 4, "ps": 64, "layout": "head"},
        # four draft tokens each for eight sequences to verify
        {"name": "chunk_draft", "lot": 4, "op": "chunk", "act": "bf16", "n": 8, "big": 8, "new": 4,
         "ragged": False, "past": 1000, "idle": 0, "Hq": 32, "Hkv": 8, "D": 128, "cap": 0.0,
         "window": 0, "slopes": False, "ps": 16, "layout": "head"},
        # a piece of one prompt beside decoding sequences and padded entries, an odd group of
        # query heads, token-major pages
        {"name": "chunk_mixed", "lot": 5, "op": "chunk", "act": "f16", "n": 34, "big": 1, "new": 509,
         "ragged": True, "past": 4099, "idle": 2, "Hq": 24, "Hkv": 8, "D": 64, "cap": 0.0,
         "window": 0, "slopes": False, "ps": 32, "layout": "token"},
        # prompts from their first token, every head its own keys, the bias by distance
        {"name": "chunk_prompts", "lot": 6, "op": "chunk", "act": "f16", "n": 5, "big": 5, "new": 1500,
         "ragged": True, "past": 0, "idle": 0, "Hq": 8, "Hkv": 8, "D": 64, "cap": 0.0,
         "window": 0, "slopes": True, "ps": 16, "layout": "head"},
        # wide heads with capped scores and a sliding window
        {"name": "chunk_window", "lot": 7, "op": "chunk", "act": "bf16", "n": 3, "big": 3, "new": 701,
         "ragged": True, "past": 9000, "idle": 0, "Hq": 16, "Hkv": 2, "D": 256, "cap": 50.0,
         "window": 4096, "slopes": False, "ps": 16, "layout": "head"},
        # the last piece of a long document
        {"name": "chunk_2048", "lot": 8, "op": "chunk", "act": "bf16", "n": 1, "big": 1, "new": 2048,
         "ragged": False, "past": 30720, "idle": 0, "Hq": 32, "Hkv": 8, "D": 128, "cap": 0.0,
         "window": 0, "slopes": False, "ps": 64, "layout": "head"},
        # a few short prompts in the place of ended ones
        {"name": "grow_4", "op": "grow", "n": 4, "new": 70, "pages": 512, "ps": 16, "seqs": 9},
        # a full server's prompts, a large pool
        {"name": "grow_64", "op": "grow", "n": 64, "new": 4000, "pages": 40000, "ps": 16,
         "seqs": 256},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "chunk", "chunk", "chunk", "grow"])
    if op == "grow":
        n, new, ps = _log(rng, 1, 64), _log(rng, 1, 4000), rng.choice([16, 32, 64, 128])
        # now and then a pool that is too small for all of them
        most = n * -(-new // ps)
        pages = min(40000, max(64, int(most * rng.uniform(0.3, 3.0)) + rng.randint(0, 500)))
        return {"op": op, "n": n, "new": new, "pages": pages, "ps": ps, "seqs": n + rng.randint(0, 192)}
    while True:
        n = _log(rng, 1, 64)
        hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 16])
        c = {"op": op, "lot": rng.randint(0, 10 ** 6), "act": rng.choice(["f16", "bf16"]), "n": n,
             "big": rng.choice([n, n, rng.randint(0, n)]),
             "new": rng.choice([rng.randint(1, 8), _log(rng, 1, 2048), _log(rng, 16, 2048) | 1]),
             "ragged": rng.random() < 0.7, "past": rng.choice([0, _log(rng, 1, 30000), _log(rng, 1, 30000)]),
             "idle": rng.randint(0, n // 8), "Hq": hkv * g, "Hkv": hkv,
             "D": rng.choice([64, 128, 256]), "ps": rng.choice([16, 32, 64, 128]),
             "layout": rng.choice(["head", "token"])}
        c["big"] = min(c["big"], n)
        if op == "append":
            c.update({"D": rng.choice([64, 80, 96, 128, 192, 256]), "inter": rng.random() < 0.5,
                      "norm": rng.random() < 0.5, "stretch": rng.choice([1, 1, 4, 8])})
            c["rot"] = rng.choice([c["D"], 16 * rng.randint(1, c["D"] // 16)])
            big = work(listed()[2])
            if n * (c["past"] + c["new"]) > 40000:
                continue
        else:
            c.update({"cap": rng.choice([0.0, 0.0, 20.0, 50.0]),
                      "window": rng.choice([0, 0, _log(rng, 1, 8192)]),
                      "slopes": rng.random() < 0.3})
            big = work(listed()[7])
        w = work(c)
        if w["bytes"] <= big["bytes"] and w["flops"] <= max(big["flops"], 1):
            return c


# ------------------------------------------------------------------------------------ the work
def _shape(case):
    """Each entry's new tokens, the tokens before them, and whether it is a padded one: the case's
    own, for every seed."""
    rng = random.Random(case["lot"])
    new, past = [], []
    for i in range(case["n"]):
        most = case["new"] if i < case["big"] else 1
        new.append(rng.randint(max(1, most // 3), most) if case["ragged"] else most)
        past.append(rng.randint(case["past"] // 2, case["past"]) if case["ragged"] else case["past"])
    order = list(range(case["n"]))
    rng.shuffle(order)
    idle = set(rng.sample(range(case["n"]), case["idle"]))
    return [new[i] for i in order], [past[i] for i in order], [i in idle for i in range(case["n"])]


def work(case):
    c = case
    if c["op"] == "grow":
        per = -(-c["new"] // c["ps"])
        got = min(c["pages"], c["n"] * per * (2 / 3 if c["new"] > 1 else 1))
        return {"bytes": 4 * c["pages"] + 16 * got + 16 * c["n"], "flops": 0}
    entries = [(m, t) for m, t, idle in zip(*_shape(c)) if not idle]
    tokens = sum(m for m, _ in entries)
    if c["op"] == "append":
        heads = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": 4 * heads * c["D"] * tokens,
                "flops": (c["Hq"] + c["Hkv"]) * c["D"] * tokens * ((4 if c["norm"] else 0) + 3)}
    window = c["window"] or 1 << 40
    # positions that any of an entry's tokens sees, and what its tokens see one by one
    keys = sum(min(t + m, window + m - 1) for m, t in entries)
    pairs = 0
    for m, t in entries:
        below = max(0, min(m, window - t))  # tokens that see all before them
        pairs += below * t + below * (below + 1) // 2 + (m - below) * window
    return {"bytes": 4 * c["Hkv"] * c["D"] * keys + 4 * c["Hq"] * c["D"] * tokens,
            "flops": 4.0 * c["Hq"] * c["D"] * pairs}


# ------------------------------------------------------------------------------------ the inputs
class State:
    pass


def prepare(case, seed):
    s = State()
    s.c = c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "grow":
        _prepare_grow(s, c, g, seed)
    else:
        _prepare_tokens(s, c, g, seed)
    return s


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_tokens(s, c, g, seed):
    act, n, ps, Hq, Hkv, D = ACT[c["act"]], c["n"], c["ps"], c["Hq"], c["Hkv"], c["D"]
    s.new, s.past, idle = _shape(c)
    # entries in any order of the slots; padded entries name no sequence
    slots = random.Random(seed).sample(range(n + 2), n)
    s.seq = [-1 if idle[i] else slots[i] for i in range(n)]
    s.start = [0]
    for m in s.new:
        s.start.append(s.start[-1] + m)
    T = s.start[-1]
    s.seqs, s.starts = _ints(s.seq), _ints(s.start)
    lens = [0] * (n + 2)
    for i, q in enumerate(s.seq):
        if q >= 0:
            lens[q] = s.past[i] + s.new[i]
    s.lens = _ints(lens)
    cols = max(1, max(-(-m // ps) for m in lens))
    num = sum(-(-m // ps) for m in lens) + 1
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)  # recycled pages lie anywhere
    s.tables = torch.full((n + 2, cols), -1, dtype=torch.int32, device="cuda")
    at = 0
    for q, m in enumerate(lens):
        s.tables[q, :-(-m // ps)] = order[at:at + -(-m // ps)]
        at += -(-m // ps)
    # one layer's K and V planes between another layer's
    shape = (Hkv, ps, D) if c["layout"] == "head" else (ps, Hkv, D)
    planes = 4 if c["op"] == "append" else 2
    s.pool = torch.randn((planes, num) + shape, generator=g, device="cuda", dtype=act)
    s.kp, s.vp = planes - 2, planes - 1
    s.k, s.v = s.pool[s.kp], s.pool[s.vp]
    s.head_stride, s.row_stride = ps * D, D
    if c["layout"] == "token":
        s.k, s.v = s.k.transpose(1, 2), s.v.transpose(1, 2)
        s.head_stride, s.row_stride = D, Hkv * D
    if c["op"] == "append":
        # a row of the qkv product: queries, keys, values
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda").to(act)
        s.q, s.nk, s.nv = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s.qw = s.kw = None
        if c["norm"]:
            s.qw = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(act)
            s.kw = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(act)
        s.freqs = _frequencies(c)
        s.f64 = torch.tensor(s.freqs, dtype=torch.float64, device="cuda")
        s.out = torch.zeros((T, Hq, D), dtype=act, device="cuda")
        if own:
            from block_scaled_bit_gb300 import bsgemv
            s.rope = bsgemv.RopePlan(c["act"], Hq, Hkv, D, rot=c["rot"], base=BASE,
                                     interleaved=c["inter"], linear=c["stretch"])
            s.cache = bsgemv.PageCache(planes, num, Hkv * ps * D * 2, ps, n + 2, cols)
        return
    # queries a little larger than unit: some keys stand out, as they do in trained models
    s.q = (torch.randn((T, Hq, D), generator=g, device="cuda") * 1.5).to(act)
    s.slopes = None
    if c["slopes"]:  # a geometric row of slopes over the heads
        s.slopes = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq).float()
    if own:
        from block_scaled_bit_gb300 import bsgemv
        s.plan = bsgemv.ChunkPlan(c["act"], Hq, Hkv, D, ps, max_n=n, max_T=T)
        s.out = torch.empty_like(s.q)


def _frequencies(c):
    """Radians a position of each pair, positions squeezed by the stretch."""
    return [BASE ** (-2 * i / c["rot"]) / c["stretch"] for i in range(c["rot"] // 2)]


def _prepare_grow(s, c, g, seed):
    n, ps, N = c["n"], c["ps"], c["pages"]
    rng = random.Random(seed)
    s.new = [rng.randint(max(1, c["new"] // 3), c["new"]) for _ in range(n)]
    s.start = [0]
    for m in s.new:
        s.start.append(s.start[-1] + m)
    s.seq = rng.sample(range(c["seqs"]), n)
    s.seqs, s.starts = _ints(s.seq), _ints(s.start)
    cols = -(-c["new"] // ps) + 1
    # the other slots hold sequences of their own, pages anywhere; the slots to grow hold ended ones
    used = int(N * rng.uniform(0.2, 0.5))
    order = torch.randperm(N, generator=g, device="cuda")[:used].to(torch.int32).tolist()
    table = [[-1] * cols for _ in range(c["seqs"])]
    lens = [0] * c["seqs"]
    for q in range(c["seqs"]):
        m = min(rng.randint(0, cols), len(order))
        for j in range(m):
            table[q][j] = order.pop()
        lens[q] = max(0, m * ps - rng.randint(0, ps - 1)) if m else 0
    s.tables, s.lens = _ints(table), _ints(lens)
    s.refs = torch.zeros(N, dtype=torch.int32, device="cuda")
    s.refs[s.tables[s.tables >= 0].long()] = 1
    s.pool = torch.zeros((2, N, 256), dtype=torch.uint8, device="cuda")  # (no page is copied)
    s.grown = torch.empty(n, dtype=torch.int32, device="cuda")
    if own:
        from block_scaled_bit_gb300 import bsgemv
        s.cache = bsgemv.PageCache(2, N, 256, ps, c["seqs"], cols)


# ------------------------------------------------------------------------------------ one pass
def run(state):
    s = state
    op = s.c["op"]
    if own:
        return _run_own(s, op)
    return {"append": _plain_append, "chunk": _plain_chunk, "grow": _plain_grow}[op](s, s.c)


def _run_own(s, op):
    if op == "append":
        s.cache.append(s.rope, s.pool, s.tables, s.lens, s.seqs, s.starts, s.q, s.nk, s.nv, s.out,
                       head_stride=s.head_stride, row_stride=s.row_stride, k_plane=s.kp,
                       v_plane=s.vp, q_weight=s.qw, k_weight=s.kw, eps=1e-6)
        return {"q": s.out, "pool": s.pool}
    if op == "chunk":
        s.plan.run(s.q, s.k, s.v, s.tables, s.lens, s.seqs, s.starts, s.out, cap=s.c["cap"],
                   window=s.c["window"], slopes=s.slopes)
        return s.out
    s.cache.free(s.refs, s.tables, s.lens, s.seqs)
    s.cache.grow(s.pool, s.refs, s.tables, s.lens, s.seqs, s.starts, s.grown)
    return {"refs": s.refs, "tables": s.tables, "lens": s.lens, "grown": s.grown}


def _rows(s, device="cuda"):
    """Entry and position of every row, on the device."""
    T, n = s.start[-1], s.c["n"]
    row = torch.arange(T, device=device)
    entry = torch.searchsorted(s.starts[1:], row, right=True, out_int32=True).clamp(max=n - 1)
    seq = s.seqs[entry].long()
    pos = s.lens[seq.clamp(min=0)].long() - s.starts[entry + 1].long() + row
    return seq, pos


def _plain_append(s, c):
    seq, pos = _rows(s)
    live = seq >= 0
    angle = pos[:, None].double() * s.f64
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def place(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        r = c["rot"]
        y, rest = x[..., :r], x[..., r:]
        if c["inter"]:
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = y[..., :r // 2], y[..., r // 2:]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([y, rest], -1).to(s.out.dtype)

    s.out.copy_(torch.where(live[:, None, None], place(s.q, s.qw), s.out))
    # padded rows go to a spare row after the pool's own (page num: none), by a masked copy
    page = s.tables[seq.clamp(min=0), (pos // c["ps"]).clamp(min=0)].long()
    at = pos % c["ps"]
    for plane, x in ((s.k, place(s.nk, s.kw)), (s.v, s.nv)):
        if c["idle"]:
            keep = live.nonzero().squeeze(1)
            plane[page[keep], :, at[keep]] = x[keep]
        else:
            plane[page, :, at] = x
    return {"q": s.out, "pool": s.pool}


def _plain_chunk(s, c):
    Hkv, D, ps = c["Hkv"], c["D"], c["ps"]
    G = c["Hq"] // Hkv
    out = torch.zeros_like(s.q)
    for i, seq in enumerate(s.seq):
        if seq < 0:
            continue
        m, total = s.new[i], s.past[i] + s.new[i]
        # the pages that some new token sees
        first = max(0, s.past[i] + 1 - c["window"]) // ps if c["window"] else 0
        pages = s.tables[seq, first:-(-total // ps)]
        lo = first * ps
        j = torch.arange(lo, total, device="cuda")
        pos = torch.arange(s.past[i], total, device="cuda")
        hidden = j[None] > pos[:, None]
        if c["window"]:
            hidden = hidden | (j[None] <= pos[:, None] - c["window"])
        rows = slice(s.start[i], s.start[i + 1])
        # heads together as far as their scores are of ordinary size
        step = max(1, min(Hkv, (1 << 28) // max(1, G * m * (total - lo))))
        for h in range(0, Hkv, step):
            hs = slice(h, h + step)
            k = s.k[pages, hs].transpose(0, 1).flatten(1, 2)[:, :total - lo].float()
            v = s.v[pages, hs].transpose(0, 1).flatten(1, 2)[:, :total - lo].float()
            heads = slice(h * G, (h + k.shape[0]) * G)
            q = s.q[rows, heads].float().view(m, -1, G, D).permute(1, 2, 0, 3) / math.sqrt(D)
            t = (q.flatten(1, 2) @ k.transpose(1, 2)).view(-1, G, m, total - lo)
            if c["cap"]:
                t = c["cap"] * torch.tanh(t / c["cap"])
            if c["slopes"]:
                t = t + s.slopes[heads].view(-1, G, 1, 1) * (j[None] - pos[:, None]).float()
            t = t.masked_fill(hidden, -math.inf)
            e = torch.exp(t - t.amax(-1, keepdim=True))
            o = (e.flatten(1, 2) @ v).view(-1, G, m, D) / e.sum(-1, keepdim=True)
            out[rows, heads] = o.permute(2, 0, 1, 3).reshape(m, -1, D).to(out.dtype)
    return out


def _plain_grow(s, c):
    ps, N = c["ps"], c["pages"]
    seq, cols = s.seqs.long(), s.tables.shape[1]
    col = torch.arange(cols, device="cuda")[None]
    # release what the ended sequences held
    rows = s.tables[seq]
    held = col < ((s.lens[seq] + ps - 1) // ps)[:, None]
    refs = torch.cat([s.refs, s.refs.new_zeros(1)])
    minus = torch.full((rows.numel(),), -1, device="cuda", dtype=torch.int32)
    refs.index_add_(0, torch.where(held, rows, N).reshape(-1).long(), minus)
    # entries in order: those whose pages, with the earlier entries', are there
    count = (s.starts[1:] - s.starts[:-1]).long()
    need = (count + ps - 1) // ps
    cum = torch.cumsum(need, 0)
    free = torch.cumsum(refs[:N] == 0, 0)
    fits = cum <= free[-1]
    # the r-th page wanted is the r-th free one
    rank = (cum - need)[:, None] + col + 1
    page = torch.searchsorted(free, rank.reshape(-1)).view(rank.shape).to(torch.int32)
    mine = (col < need[:, None]) & fits[:, None]
    refs.index_add_(0, torch.where(mine, page, N).reshape(-1).long(), -minus)
    s.tables[seq] = torch.where(mine, page, -1)
    s.lens[seq] = torch.where(fits, count, 0).to(torch.int32)
    s.refs.copy_(refs[:N])
    s.grown.copy_(fits)
    return {"refs": s.refs, "tables": s.tables, "lens": s.lens, "grown": s.grown}


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The computed outputs from the operators' definitions in 64 bits; what grow gives are whole
    numbers, which the plain form gives exactly."""
    if case["op"] == "grow":
        return None
    s = prepare(case, seed)
    return _exact_append(s, s.c) if case["op"] == "append" else _exact_chunk(s, s.c)


def _exact_append(s, c):
    pool, q = s.pool.double(), torch.zeros(s.out.shape, dtype=torch.float64, device="cuda")
    planes = [pool[s.kp], pool[s.vp]]
    if c["layout"] == "token":
        planes = [x.transpose(1, 2) for x in planes]
    half, D = c["rot"] // 2, c["D"]
    # the two places of each pair
    pair = torch.arange(half, device="cuda")
    first = 2 * pair if c["inter"] else pair
    second = first + 1 if c["inter"] else pair + half

    def turned(x, w, pos):
        y = x.double()
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        z = y.clone()
        phase = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[:, None] * s.f64)
        both = torch.complex(y[..., first], y[..., second]) * phase[:, None]
        z[..., first], z[..., second] = both.real, both.imag
        return z

    for i, seq in enumerate(s.seq):
        if seq < 0:
            continue
        at = torch.arange(s.past[i], s.past[i] + s.new[i], device="cuda")
        rows = slice(s.start[i], s.start[i + 1])
        q[rows] = turned(s.q[rows], s.qw, at.double())
        page, row = s.tables[seq].long()[at // c["ps"]], at % c["ps"]
        planes[0][page, :, row] = turned(s.nk[rows], s.kw, at.double())
        planes[1][page, :, row] = s.nv[rows].double()
    return {"q": q, "pool": pool}


def _exact_chunk(s, c):
    D, G = c["D"], c["Hq"] // c["Hkv"]
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    for i, seq in enumerate(s.seq):
        if seq < 0:
            continue
        m, total = s.new[i], s.past[i] + s.new[i]
        pages = s.tables[seq, :-(-total // c["ps"])].long()
        i0 = torch.arange(s.past[i], total, device="cuda")[:, None]
        j0 = torch.arange(total, device="cuda")[None]
        seen = (j0 <= i0) & ((j0 > i0 - c["window"]) if c["window"] else (j0 >= 0))
        for h in range(c["Hq"]):
            k = s.k[pages, h // G].reshape(-1, D)[:total].double()
            v = s.v[pages, h // G].reshape(-1, D)[:total].double()
            t = (s.q[s.start[i]:s.start[i + 1], h].double() @ k.T) * D ** -0.5
            if c["cap"]:
                t = torch.tanh(t / c["cap"]) * c["cap"]
            if c["slopes"]:
                t = t - s.slopes[h].double() * (i0 - j0)
            t = torch.where(seen, t, -math.inf)
            out[s.start[i]:s.start[i + 1], h] = torch.softmax(t, -1) @ v
    return out
