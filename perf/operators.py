"""The decode-step operators around the block-scaled GEMV, as cases that can be timed and compared.

Three operators, each in a plain form (elementary torch operations in fp32, rounded once) and as
the calls a program makes of the library:

  moe    a whole mixture-of-experts layer for a few tokens: top-k routing of the router's logits,
         the chosen experts' gate and up products, SiLU(gate) * up, the down product and the
         weighted sum, with expert weights in the library's four block-scaled formats
  attn   single-token attention of a batch whose sequences share a long prefix, over a paged cache
  fork,  the pages of that cache: sequences forked from a prompt (full pages shared, the partial
  compact  page copied), and live pages moved down to close the holes

`own` selects the side: False the plain form, True the library.
"""
import math

import torch

own = False

ACT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one user decoding, many small experts: eight experts' weights are read, latency counts
        {"name": "moe_int4_1", "op": "moe", "fmt": "int4", "act": "f16", "bs": 32, "zp": False,
         "H": 2048, "I": 512, "E": 256, "k": 8, "T": 1},
        # a small batch on NVFP4 experts
        {"name": "moe_nvfp4_8", "op": "moe", "fmt": "nvfp4", "act": "bf16", "bs": 16, "zp": False,
         "H": 2048, "I": 768, "E": 128, "k": 8, "T": 8},
        # sizes that are no multiple of the k or row tiles, zero points, few experts: most experts
        # serve several tokens
        {"name": "moe_int8_13", "op": "moe", "fmt": "int8", "act": "bf16", "bs": 32, "zp": True,
         "H": 2752, "I": 960, "E": 48, "k": 4, "T": 13},
        # the largest batch: nearly every FP8 expert is read, with three tokens on average
        {"name": "moe_fp8_32", "op": "moe", "fmt": "fp8", "act": "bf16", "bs": 128, "zp": False,
         "H": 4096, "I": 1408, "E": 64, "k": 6, "T": 32},
        # one sequence after a short system prompt
        {"name": "attn_1", "op": "attn", "act": "bf16", "B": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "ps": 16, "P": 512, "own_max": 60, "idle": 0, "layout": "head"},
        # a prefix that ends inside a page, an odd group of query heads, token-major pages
        {"name": "attn_odd_16", "op": "attn", "act": "f16", "B": 16, "Hq": 24, "Hkv": 8, "D": 64,
         "ps": 32, "P": 4099, "own_max": 700, "idle": 1, "layout": "token"},
        # wide heads, idle slots among the sequences
        {"name": "attn_d256_48", "op": "attn", "act": "bf16", "B": 48, "Hq": 16, "Hkv": 2,
         "D": 256, "ps": 16, "P": 16384, "own_max": 300, "idle": 5, "layout": "head"},
        # a full batch over a long shared document
        {"name": "attn_64", "op": "attn", "act": "bf16", "B": 64, "Hq": 32, "Hkv": 8, "D": 128,
         "ps": 64, "P": 32768, "own_max": 1024, "idle": 0, "layout": "head"},
        # four samples of one short prompt
        {"name": "fork_4", "op": "fork", "planes": 8, "pages": 512, "page_bytes": 8192, "ps": 16,
         "plen": 1003, "n": 4, "table": 128},
        # sixty-four samples of a long prompt
        {"name": "fork_64", "op": "fork", "planes": 16, "pages": 1536, "page_bytes": 65536,
         "ps": 32, "plen": 32775, "n": 64, "table": 1280},
        # a small pool after a few sequences have ended
        {"name": "compact_small", "op": "compact", "planes": 8, "pages": 300, "page_bytes": 8192,
         "ps": 16, "seqs": 7, "live": 0.5, "table": 64},
        # a large pool, half of it live
        {"name": "compact_large", "op": "compact", "planes": 16, "pages": 2048,
         "page_bytes": 65536, "ps": 32, "seqs": 33, "live": 0.5, "table": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["moe", "moe", "attn", "attn", "fork", "compact"])
    if op == "moe":
        fmt = rng.choice(["int4", "int8", "fp8", "nvfp4"])
        bs = {"fp8": 128, "nvfp4": 16}.get(fmt) or rng.choice([16, 32, 64, 128])
        step = max(64, bs)
        big = work(listed()[3])["bytes"]
        while True:
            c = {"op": op, "fmt": fmt, "act": rng.choice(["f16", "bf16"]), "bs": bs,
                 "zp": fmt in ("int4", "int8") and rng.random() < 0.5,
                 "H": rng.choice([2 ** rng.randint(8, 12), step * (_log(rng, 256, 4032) // step | 1)]),
                 "I": step * max(1, _log(rng, 128, 1472) // step),
                 "E": _log(rng, 4, 256), "T": _log(rng, 1, 32)}
            c["k"] = rng.randint(1, min(8, c["E"]))
            if work(c)["bytes"] <= big:
                return c
    if op == "attn":
        big = work(listed()[7])
        while True:
            hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 16])
            b = _log(rng, 1, 64)
            c = {"op": op, "act": rng.choice(["f16", "bf16"]), "B": b, "Hq": hkv * g, "Hkv": hkv,
                 "D": rng.choice([64, 128, 256]), "ps": rng.choice([16, 32, 64, 128]),
                 "P": rng.choice([0, 2 ** rng.randint(4, 15), _log(rng, 16, 32767) | 1]), "own_max": _log(rng, 1, 1500),
                 "idle": rng.randint(0, b // 8), "layout": rng.choice(["head", "token"])}
            w = work(c)
            if w["bytes"] <= big["bytes"] and w["flops"] <= big["flops"]:
                return c
    ps = rng.choice([16, 32, 64])
    planes = rng.choice([2, 4, 8, 12, 16])
    page_bytes = 16 * (_log(rng, 64, 4095) | 1)
    if op == "fork":
        n, plen = _log(rng, 1, 64), _log(rng, 1, 32800) | 1
        full = -(-plen // ps)
        return {"op": op, "planes": planes, "pages": full + n + rng.randint(0, 200),
                "page_bytes": page_bytes, "ps": ps, "plen": plen, "n": n,
                "table": full + rng.randint(1, 64)}
    pages = _log(rng, 64, 2048)
    seqs = rng.randint(1, 33)
    return {"op": op, "planes": planes, "pages": pages, "page_bytes": page_bytes, "ps": ps,
            "seqs": seqs, "live": rng.uniform(0.1, 0.9), "table": pages}


# ------------------------------------------------------------------------------------ the work
def _weight_bytes(c, rows, k):
    """Bytes of one [rows, k] weight with its scales and zero points."""
    code = rows * k // (2 if c["fmt"] in ("int4", "nvfp4") else 1)
    nb = k // c["bs"]
    scale = rows * nb * {"int4": 2, "int8": 2, "fp8": 4, "nvfp4": 1}[c["fmt"]]
    zp = 0
    if c["zp"]:
        zp = rows * ((nb + 1) // 2 if c["fmt"] == "int4" else nb)
    return code + scale + zp


def work(case):
    c = case
    if c["op"] == "moe":
        # experts that uniform routing is expected to touch; their weights are read once
        active = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])
        per = _weight_bytes(c, 2 * c["I"], c["H"]) + _weight_bytes(c, c["H"], c["I"])
        return {"bytes": active * per + 4 * c["T"] * c["H"] + 2 * c["T"] * c["E"],
                "flops": 6.0 * c["T"] * c["k"] * c["H"] * c["I"]}
    if c["op"] == "attn":
        own_tokens = (c["B"] - c["idle"]) * (c["own_max"] + 1) / 2
        kv = 2 * 2 * c["Hkv"] * c["D"]
        return {"bytes": (c["P"] + own_tokens) * kv + 4 * c["B"] * c["Hq"] * c["D"],
                "flops": 4.0 * c["Hq"] * c["D"] * ((c["B"] - c["idle"]) * c["P"] + own_tokens)}
    if c["op"] == "fork":
        part = 1 if c["plen"] % c["ps"] else 0
        return {"bytes": 2 * part * c["n"] * c["planes"] * c["page_bytes"] + 8 * c["n"] * c["table"]
                + 8 * c["pages"], "flops": 0}
    live = int(c["pages"] * c["live"])
    moved = live * (1 - live / c["pages"])
    return {"bytes": 2 * moved * c["planes"] * c["page_bytes"] + 8 * c["pages"]
            + 8 * c["seqs"] * c["table"], "flops": 0}


# ------------------------------------------------------------------------------------ the inputs
class State:
    pass


def prepare(case, seed):
    c = dict(case)
    s = State()
    s.c = c
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    {"moe": _prepare_moe, "attn": _prepare_attn, "fork": _prepare_fork,
     "compact": _prepare_compact}[c["op"]](s, c, g)
    return s


def _uniform(g, shape, lo, hi):
    return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo


def _bytes(g, shape, lo=0, hi=256):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.uint8)


def _weights(g, c, rows, k):
    """Codes, scales and zero points of E stacked [rows, k] weights, in the library's layouts."""
    E, nb = c["E"], k // c["bs"]
    if c["fmt"] == "int4":
        zp = _bytes(g, (E, rows, (nb + 1) // 2)) if c["zp"] else None
        return _bytes(g, (E, rows, k // 2)), _uniform(g, (E, rows, nb), 0.005, 0.02).half(), zp
    if c["fmt"] == "int8":
        zp = _bytes(g, (E, rows, nb), 120, 137) if c["zp"] else None
        return _bytes(g, (E, rows, k)), _uniform(g, (E, rows, nb), 0.0003, 0.0012).half(), zp
    if c["fmt"] == "fp8":
        w = torch.randn((E, rows, k), generator=g, device="cuda", dtype=torch.bfloat16)
        w = (w * 64).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return w, _uniform(g, (E, rows, nb), 0.15, 0.6) / 448, None
    # NVFP4: E4M3 scale codes of [2^-4, 2^4], one fp32 global scale for each expert
    return _bytes(g, (E, rows, k // 2)), _bytes(g, (E, rows, nb), 0x18, 0x59), \
        _uniform(g, (E,), 0.8, 1.2) / 512


def _prepare_moe(s, c, g):
    act = ACT[c["act"]]
    s.x = torch.randn((c["T"], c["H"]), generator=g, device="cuda").to(act)
    s.logits = (torch.randn((c["T"], c["E"]), generator=g, device="cuda") * 2).to(act)
    s.w13, s.s13, s.z13 = _weights(g, c, 2 * c["I"], c["H"])
    s.w2, s.s2, s.z2 = _weights(g, c, c["H"], c["I"])
    if own:
        from block_scaled_bit_gb300 import bsgemv
        s.plan = bsgemv.MoePlan(c["fmt"], c["act"], c["bs"], c["zp"], c["H"], c["I"], c["E"],
                                c["k"], max_T=c["T"])
        s.y = torch.empty_like(s.x)


def _prepare_attn(s, c, g):
    act, B, ps, P = ACT[c["act"]], c["B"], c["ps"], c["P"]
    # lengths: the prefix plus 1 .. own_max tokens of a sequence's own; idle slots are empty
    lens = P + torch.randint(1, c["own_max"] + 1, (B,), generator=g, device="cuda")
    idle = torch.randperm(B, generator=g, device="cuda")[:c["idle"]]
    lens[idle] = 0
    shared = P // ps  # whole pages of the prefix; a page that it ends in is each sequence's own
    own_pages = (P + c["own_max"] + ps - 1) // ps - shared
    cols = shared + own_pages
    tail = 1 if P % ps else 0
    num = shared + tail + B * own_pages
    order = torch.randperm(num, generator=g, device="cuda")  # recycled pages lie anywhere
    pre = order[:shared + tail]
    mine = order[shared + tail:].view(B, own_pages)
    s.prefix_table = pre.to(torch.int32)
    s.tables = torch.cat([pre[:shared].expand(B, shared), mine], 1).to(torch.int32).contiguous()
    assert s.tables.shape == (B, cols)
    s.lens, s.P = lens.to(torch.int32), P
    shape = (num, c["Hkv"], ps, c["D"]) if c["layout"] == "head" else (num, ps, c["Hkv"], c["D"])
    s.k = torch.randn(shape, generator=g, device="cuda", dtype=act)
    s.v = torch.randn(shape, generator=g, device="cuda", dtype=act)
    if c["layout"] == "token":  # the views are [page, head, token, D] either way
        s.k, s.v = s.k.transpose(1, 2), s.v.transpose(1, 2)
    if tail:  # each sequence's copy of the page that the prefix ends in
        s.k[mine[:, 0], :, :P % ps] = s.k[pre[-1], :, :P % ps].unsqueeze(0)
        s.v[mine[:, 0], :, :P % ps] = s.v[pre[-1], :, :P % ps].unsqueeze(0)
    # queries a little larger than unit: some keys stand out, as they do in trained models
    s.q = (torch.randn((B, c["Hq"], c["D"]), generator=g, device="cuda") * 1.5).to(act)
    if own:
        from block_scaled_bit_gb300 import bsgemv
        s.plan = bsgemv.AttnPlan(c["act"], c["Hq"], c["Hkv"], c["D"], ps, max_B=B)
        s.out = torch.empty_like(s.q)


def _plane_words(c):
    return c["page_bytes"] // 2


def _pool(s, c, g):
    s.pool = torch.randint(-32768, 32767, (c["planes"], c["pages"], _plane_words(c)), generator=g,
                           device="cuda", dtype=torch.int16)


def _cache(s, c, seqs):
    if own:
        from block_scaled_bit_gb300 import bsgemv
        s.cache = bsgemv.PageCache(c["planes"], c["pages"], c["page_bytes"], c["ps"], seqs,
                                   c["table"])


def _prepare_fork(s, c, g):
    _pool(s, c, g)
    n, full = c["n"], -(-c["plen"] // c["ps"])
    pages = torch.randperm(c["pages"], generator=g, device="cuda")[:full]
    # the prompt sits in one slot, its samples go to the others
    at = torch.randperm(n + 1, generator=g, device="cuda")
    s.tables = torch.full((n + 1, c["table"]), -1, device="cuda", dtype=torch.int32)
    s.lens = torch.zeros(n + 1, device="cuda", dtype=torch.int32)
    s.tables[at[0], :full] = pages.to(torch.int32)
    s.lens[at[0]] = c["plen"]
    s.refs = torch.zeros(c["pages"], device="cuda", dtype=torch.int32)
    s.refs[pages] = 1
    s.parents = at[:1].expand(n).to(torch.int32).contiguous()
    s.children = at[1:].to(torch.int32).contiguous()
    s.new = torch.empty(n, device="cuda", dtype=torch.int32)
    _cache(s, c, n + 1)


def _prepare_compact(s, c, g):
    _pool(s, c, g)
    S, live = c["seqs"], max(1, int(c["pages"] * c["live"]))
    pages = torch.randperm(c["pages"], generator=g, device="cuda")[:live].to(torch.int32)
    # the live pages dealt out to the sequences; every sequence shares page 0 of the deal
    col = torch.arange(c["table"], device="cuda")
    per = (live - 1) // S
    count = torch.randint(0, per + 1, (S,), generator=g, device="cuda").clamp_(max=c["table"] - 1)
    start = 1 + per * torch.arange(S, device="cuda")
    src = torch.where(col[None] == 0, 0, start[:, None] + col[None] - 1)
    used = col[None] <= count[:, None]
    s.tables = torch.where(used, pages[src.clamp(max=live - 1)], -1).to(torch.int32)
    s.lens = ((count + 1) * c["ps"]).to(torch.int32)
    s.refs = torch.zeros(c["pages"] + 1, device="cuda", dtype=torch.int32)
    s.refs.index_add_(0, torch.where(used, s.tables, c["pages"]).reshape(-1).long(),
                      torch.ones(s.tables.numel(), device="cuda", dtype=torch.int32))
    s.refs = s.refs[:c["pages"]].clone()
    s.refs_out, s.tables_out = torch.empty_like(s.refs), torch.empty_like(s.tables)
    s.live = torch.empty(1, device="cuda", dtype=torch.int32)
    _cache(s, c, S)


# ------------------------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        return _run_own(s, s.c["op"])
    return {"moe": _plain_moe, "attn": _plain_attn, "fork": _plain_fork,
            "compact": _plain_compact}[s.c["op"]](s, s.c)


def _run_own(s, op):
    if op == "moe":
        s.plan.run(s.x, s.logits, s.w13, s.s13, s.z13, s.w2, s.s2, s.z2, s.y)
        return s.y
    if op == "attn":
        s.plan.run(s.q, s.k, s.v, s.prefix_table, s.P, s.tables, s.lens, s.out)
        return s.out
    if op == "fork":
        s.cache.fork(s.pool, s.refs, s.tables, s.lens, s.parents, s.children, s.new)
        return {"pool": s.pool, "refs": s.refs, "tables": s.tables, "lens": s.lens, "new": s.new}
    s.cache.compact(s.pool, s.refs, s.tables, s.lens, s.refs_out, s.tables_out, s.live)
    return {"pool": s.pool, "refs": s.refs_out, "tables": s.tables_out, "live": s.live}


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nibbles(w):
    return torch.stack([w & 15, w >> 4], -1).flatten(-2)


def _dequant(c, w, sc, zp):
    """[..., rows, k] fp32 weights from codes, scales and zero points (zp: the global scales of
    these experts for NVFP4)."""
    if c["fmt"] == "nvfp4":
        table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=w.device)
        q = table[_nibbles(w).int()]
        sc = sc.view(torch.float8_e4m3fn).float() * zp[..., None, None]
    elif c["fmt"] == "fp8":
        q, sc = w.view(torch.float8_e4m3fn).float(), sc.float()
    else:
        q = (_nibbles(w) if c["fmt"] == "int4" else w).float()
        sc = sc.float()
        if zp is not None:
            z = (_nibbles(zp)[..., :sc.shape[-1]] if c["fmt"] == "int4" else zp).float()
        else:
            z = torch.full_like(sc, 8.0 if c["fmt"] == "int4" else 128.0)
        return ((q.unflatten(-1, (-1, c["bs"])) - z[..., None]) * sc[..., None]).flatten(-2)
    return (q.unflatten(-1, (-1, c["bs"])) * sc[..., None]).flatten(-2)


def _plain_moe(s, c):
    # a stable sort gives the lowest expert where logits tie
    top, ids = torch.sort(s.logits.float(), dim=-1, descending=True, stable=True)
    top, ids = top[:, :c["k"]], ids[:, :c["k"]]
    p = torch.exp(top - top[:, :1])
    p = p / p.sum(-1, keepdim=True)
    pick = lambda t: None if t is None else t[ids]  # noqa: E731
    w13 = _dequant(c, pick(s.w13), pick(s.s13), pick(s.z13))      # [T, k, 2I, H]
    gu = (w13 @ s.x.float()[:, None, :, None]).squeeze(-1)
    gate, up = gu[..., :c["I"]], gu[..., c["I"]:]
    h = gate / (1 + torch.exp(-gate)) * up * p[..., None]
    w2 = _dequant(c, pick(s.w2), pick(s.s2), pick(s.z2))          # [T, k, H, I]
    return (w2 @ h[..., None]).squeeze(-1).sum(1).to(s.x.dtype)


def _plain_attn(s, c):
    B, Hkv, D, ps, P = c["B"], c["Hkv"], c["D"], c["ps"], s.P
    G = c["Hq"] // Hkv
    q = s.q.float().view(B, Hkv, G, D) / math.sqrt(D)
    # the prefix, read once for all: [Hkv, P, D]
    kp = s.k[s.prefix_table].transpose(0, 1).flatten(1, 2)[:, :P].float()
    vp = s.v[s.prefix_table].transpose(0, 1).flatten(1, 2)[:, :P].float()
    sp = torch.einsum("bhgd,hpd->bhgp", q, kp)
    # the sequences' own tokens, padded to the longest
    first = P // ps
    mine = s.tables[:, first:]
    pos = first * ps + torch.arange(mine.shape[1] * ps, device=q.device)
    valid = (pos[None] >= P) & (pos[None] < s.lens[:, None])
    ko = s.k[mine].transpose(1, 2).flatten(2, 3).float()          # [B, Hkv, own, D]
    vo = s.v[mine].transpose(1, 2).flatten(2, 3).float()
    so = torch.einsum("bhgd,bhpd->bhgp", q, ko)
    so = torch.where(valid[:, None, None], so, -math.inf)
    score = torch.cat([sp, so], -1)
    e = torch.exp(score - score.max(-1, keepdim=True).values)
    e = e / e.sum(-1, keepdim=True)
    o = torch.einsum("bhgp,hpd->bhgd", e[..., :P], vp) + torch.einsum("bhgp,bhpd->bhgd", e[..., P:], vo)
    here = (s.lens >= max(P, 1))[:, None, None]  # an idle slot attends to nothing
    return torch.where(here, o.reshape(B, c["Hq"], D), 0.0).to(s.q.dtype)


def _plain_fork(s, c):
    ps, N = c["ps"], c["pages"]
    col = torch.arange(c["table"], device="cuda")[None]
    rows, old = s.tables[s.parents], s.tables[s.children]
    plen = s.lens[s.parents]
    full, part = plen // ps, plen % ps > 0
    shared = col < full[:, None]
    held = col < ((s.lens[s.children] + ps - 1) // ps)[:, None]
    # share the full pages, release what the children held
    refs = torch.cat([s.refs, s.refs.new_zeros(1)])
    one = torch.ones(rows.numel(), device="cuda", dtype=torch.int32)
    refs.index_add_(0, torch.where(shared, rows, N).reshape(-1), one)
    refs.index_add_(0, torch.where(held, old, N).reshape(-1), -one)
    # the r-th child that needs a page of its own takes the r-th free page, lowest first
    rank = torch.cumsum(part, 0)
    free = torch.cumsum(refs[:N] == 0, 0)
    new = torch.searchsorted(free, rank).to(torch.int32)
    new = torch.where(part, new, -1)
    last = rows.gather(1, full.clamp(max=c["table"] - 1)[:, None].long()).squeeze(1)
    src, dst = torch.where(part, last, 0), torch.where(part, new, 0)
    s.pool[:, dst] = s.pool[:, src]
    refs.index_add_(0, torch.where(part, new, N), one[:c["n"]])
    row = torch.where(shared, rows, -1)
    row = torch.where((col == full[:, None]) & part[:, None], new[:, None], row)
    s.tables[s.children] = row
    s.lens[s.children] = plen
    s.refs.copy_(refs[:N])
    return {"pool": s.pool, "refs": s.refs, "tables": s.tables, "lens": s.lens, "new": new}


def _plain_compact(s, c):
    at = torch.arange(c["pages"], device="cuda", dtype=torch.int32)
    live = s.refs > 0
    count = live.sum().to(torch.int32)
    hole = (~live & (at < count)).nonzero().squeeze(1)
    mover = (live & (at >= count)).nonzero().squeeze(1)
    s.pool[:, hole] = s.pool[:, mover]
    to = at.clone()
    to[mover] = at[hole]
    tables = torch.where(s.tables >= 0, to[s.tables.clamp(min=0)], -1)
    refs = s.refs.clone()
    refs[hole] = s.refs[mover]
    refs[mover] = 0
    return {"pool": s.pool, "refs": refs, "tables": tables, "live": count.view(1)}


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The computed outputs from the operators' definitions in 64 bits; the cache operators'
    outputs are whole numbers, which the plain form gives exactly."""
    s = prepare(case, seed)
    if case["op"] == "moe":
        return _exact_moe(s, s.c)
    return _exact_attn(s, s.c) if case["op"] == "attn" else None


def _e4m3_table():
    vals = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v = math.nan if code & 127 == 127 else v
        vals.append(-v if code & 128 else v)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _weight64(c, w, sc, zp, e):
    """Expert e's weight, element by element of its definition."""
    w, sc = w[e], sc[e]
    rows, nb = sc.shape
    if c["fmt"] in ("int4", "nvfp4"):
        code = torch.empty((rows, 2 * w.shape[1]), dtype=torch.int64, device="cuda")
        code[:, 0::2], code[:, 1::2] = (w % 16).long(), (w // 16).long()
    else:
        code = w.long()
    if c["fmt"] == "nvfp4":
        mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        value = mag[code % 8] * (1 - 2 * (code // 8)).double()
        scale = _e4m3_table()[sc.long()] * zp[e].double()
    elif c["fmt"] == "fp8":
        value, scale = _e4m3_table()[code], sc.double()
    else:
        z = torch.full((rows, nb), 8 if c["fmt"] == "int4" else 128, dtype=torch.int64, device="cuda")
        if zp is not None and c["fmt"] == "int8":
            z = zp[e].long()
        elif zp is not None:
            for b in range(nb):
                z[:, b] = (zp[e][:, b // 2].long() >> (4 * (b % 2))) & 15
        value, scale = (code - z.repeat_interleave(c["bs"], 1)).double(), sc.double()
    return value * scale.repeat_interleave(c["bs"], 1)


def _exact_moe(s, c):
    x, y = s.x.double(), torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
    chosen = {}
    for t, row in enumerate(s.logits.double().tolist()):
        best = sorted(range(c["E"]), key=lambda e: (-row[e], e))[:c["k"]]
        total = sum(math.exp(row[e] - row[best[0]]) for e in best)
        for e in best:
            chosen.setdefault(e, []).append((t, math.exp(row[e] - row[best[0]]) / total))
    for e, users in chosen.items():
        w13, w2 = _weight64(c, s.w13, s.s13, s.z13, e), _weight64(c, s.w2, s.s2, s.z2, e)
        for t, p in users:
            gu = w13 @ x[t]
            gate, up = gu[:c["I"]], gu[c["I"]:]
            y[t] += p * (w2 @ (gate * torch.sigmoid(gate) * up))
    return y


def _exact_attn(s, c):
    B, Hkv, D, ps, P = c["B"], c["Hkv"], c["D"], c["ps"], s.P
    G = c["Hq"] // Hkv
    out = torch.zeros((B, c["Hq"], D), dtype=torch.float64, device="cuda")
    lens = s.lens.tolist()
    for h in range(Hkv):
        kp = torch.cat([s.k[p, h] for p in s.prefix_table.tolist()])[:P].double() if P else None
        vp = torch.cat([s.v[p, h] for p in s.prefix_table.tolist()])[:P].double() if P else None
        for b in range(B):
            if lens[b] < max(P, 1):
                continue
            pages = s.tables[b, P // ps:].long()
            lo, hi = P % ps, lens[b] - P // ps * ps
            k = s.k[pages, h].reshape(-1, D)[lo:hi].double()
            v = s.v[pages, h].reshape(-1, D)[lo:hi].double()
            q = s.q[b, h * G:(h + 1) * G].double()
            score = q @ (k if kp is None else torch.cat([kp, k])).T * D ** -0.5
            out[b, h * G:(h + 1) * G] = torch.softmax(score, -1) @ (v if vp is None else torch.cat([vp, v]))
    return out
