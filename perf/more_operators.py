"""Cases of a prompt's way into the paged cache: pages and slots for new tokens
(release and assign), rotary positions applied to queries and keys on their way
into the pool, and attention of the new tokens over the cache.

`run` computes each operator in elementary torch operations (32-bit, angles in
64), or, with `own` set, through the library's calls.  `exact` computes the same
outputs from the definitions in 64 bits.

Pages.  Bit p % 32 of word p / 32 of `free` is 1 where page p is free.  A step
gives back the pages behind every request's length, then gives each request the
pages its new tokens need, the lowest free ones in request order.  Token i of
request b has position len_b + i and slot table[b, position / page] * page +
position % page.

Rotary positions.  Pair i of the first R elements of a head turns by position *
freq_i: elements (2 i, 2 i + 1) interleaved, (i, i + R / 2) in halves.

Chunk attention.  Row i of request b's n_b new tokens stands at position p =
len_b - n_b + i (len_b counts them) and attends to tokens max(0, p - W + 1) .. p
(W = 0: from the first).
"""
import math

import torch

own = False

D = 128
PAGE = 16  # the page size of the repository's workloads


def listed():
    return [
        # one decode step of a serving batch, one token each: latency
        {"name": "pages_step", "op": "pages", "batch": 64, "new_lo": 1, "new_hi": 1, "past_lo": 16, "past_hi": 4096, "page": PAGE},
        # a wave of ragged prompts, some behind earlier turns
        {"name": "pages_prompts", "op": "pages", "batch": 300, "new_lo": 1, "new_hi": 1500, "past_lo": 0, "past_hi": 8192, "page": PAGE},
        # one decode step of a serving batch, 32 / 8 heads: latency
        {"name": "rope_step", "op": "rope", "batch": 64, "hkv": 8, "g": 4, "new_lo": 1, "new_hi": 1, "past_lo": 16, "past_hi": 4096, "page": PAGE, "dtype": "bf16",
         "kind": "bf16", "rot": 128, "inter": False, "factor": 1.0},
        # ragged prompts at far positions of a context stretched eight times
        {"name": "rope_prompts", "op": "rope", "batch": 24, "hkv": 8, "g": 4, "new_lo": 1, "new_hi": 4096, "past_lo": 0, "past_hi": 120000, "page": PAGE,
         "dtype": "f16", "kind": "f16", "rot": 128, "inter": True, "factor": 8.0},
        # half of each head rotated, an fp8 cache, one query head per KV head
        {"name": "rope_part_e4m3", "op": "rope", "batch": 7, "hkv": 32, "g": 1, "new_lo": 1, "new_hi": 700, "past_lo": 0, "past_hi": 5000, "page": PAGE,
         "dtype": "f16", "kind": "e4m3", "rot": 64, "inter": False, "factor": 1.0},
        # a small interactive batch, a few tokens each: latency
        {"name": "chunk_tiny", "op": "chunk", "batch": 4, "hkv": 32, "g": 1, "new_lo": 1, "new_hi": 4, "ones": False, "past_lo": 32, "past_hi": 300, "window": 0,
         "page": PAGE, "dtype": "f16"},
        # prompts from the start, ragged, 32 / 8 heads
        {"name": "chunk_prompts", "op": "chunk", "batch": 8, "hkv": 8, "g": 4, "new_lo": 900, "new_hi": 4096, "ones": False, "past_lo": 0, "past_hi": 0,
         "window": 0, "page": PAGE, "dtype": "bf16"},
        # a chunk of a long document
        {"name": "chunk_long", "op": "chunk", "batch": 1, "hkv": 8, "g": 4, "new_lo": 2047, "new_hi": 2047, "ones": False, "past_lo": 65001, "past_hi": 65001,
         "window": 0, "page": PAGE, "dtype": "bf16"},
        # a mixed step: most requests decode one token, some bring a chunk
        {"name": "chunk_mixed", "op": "chunk", "batch": 64, "hkv": 8, "g": 4, "new_lo": 333, "new_hi": 512, "ones": True, "past_lo": 100, "past_hi": 4096,
         "window": 0, "page": PAGE, "dtype": "f16"},
        # speculated tokens of two long requests: the work is split over the cache
        {"name": "chunk_spec", "op": "chunk", "batch": 2, "hkv": 4, "g": 8, "new_lo": 5, "new_hi": 5, "ones": False, "past_lo": 100001, "past_hi": 131072,
         "window": 0, "page": PAGE, "dtype": "bf16"},
        # a sliding window over a long prompt, one query head per KV head
        {"name": "chunk_window", "op": "chunk", "batch": 2, "hkv": 16, "g": 1, "new_lo": 5000, "new_hi": 8192, "ones": False, "past_lo": 0, "past_hi": 2000,
         "window": 1024, "page": 64, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("pages", "rope", "rope", "chunk", "chunk", "chunk"))
    page = rng.choice((8, 16, 16, 32, 64, 20))
    if op == "pages":
        hi = _log_int(rng, 1, 4096)
        batch = _log_int(rng, 1, max(1, min(512, (1 << 18) // hi)))
        return {"op": op, "batch": batch, "new_lo": rng.choice((0, 1, hi)), "new_hi": hi, "past_lo": 0, "past_hi": _log_int(rng, 1, 8192), "page": page}
    hkv, g = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 8))
    dtype = rng.choice(("f16", "bf16"))
    if op == "rope":
        hi = _log_int(rng, 1, 4096)
        batch = _log_int(rng, 1, max(1, min(200, 32768 // hi)))
        return {"op": op, "batch": batch, "hkv": hkv, "g": g, "new_lo": 1, "new_hi": hi, "past_lo": 0, "past_hi": _log_int(rng, 1, 120000), "page": page,
                "dtype": dtype, "kind": rng.choice((dtype, dtype, "e4m3")), "rot": rng.choice((32, 64, 96, 128, 128)), "inter": rng.random() < 0.5,
                "factor": rng.choice((1.0, 4.0, 8.0))}
    new = _log_int(rng, 1, 4096)
    past = _log_int(rng, 1, max(1, min(65536, (1 << 26) // (new * hkv * g))))
    most = max(1, min(64, (1 << 27) // (hkv * g * new * (new + past)), (1 << 19) // (new + past)))
    return {"op": op, "batch": _log_int(rng, 1, most), "hkv": hkv, "g": g, "new_lo": rng.choice((1, max(1, new // 2))), "new_hi": new,
            "ones": rng.random() < 0.2, "past_lo": rng.choice((0, past)), "past_hi": past, "window": rng.choice((0, 0, 0, _log_int(rng, 1, 4096))),
            "page": page, "dtype": dtype}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _lengths(case):
    """New and earlier tokens of each request: the case's own, so that its outputs have one shape for every seed."""
    b = case["batch"]
    gen = torch.Generator().manual_seed(12345 + b + case["new_hi"])
    new = torch.randint(case["new_lo"], case["new_hi"] + 1, (b,), generator=gen, dtype=torch.int32)
    past = torch.randint(case["past_lo"], case["past_hi"] + 1, (b,), generator=gen, dtype=torch.int32)
    if case.get("ones"):
        new = torch.where(torch.arange(b) % 16 == b // 2 % 16, new, torch.ones_like(new))
    return new, past


def _indptr(new):
    out = torch.zeros(len(new) + 1, dtype=torch.int32)
    out[1:] = torch.cumsum(new, 0)
    return out


def _tables(lens, page, gen, extra):
    """Block table [B, max pages] (-1 unused) over a permuted pool of `extra` more pages than are used, and the pool's pages."""
    need = (lens.long() + page - 1) // page
    used, width = int(need.sum()), max(1, int(need.max()))
    perm = torch.randperm(used + extra, generator=gen).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    mine = torch.arange(width)[None, :] < need[:, None]
    table[mine] = perm[:used]
    return table, used + extra


def _normal(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device=gen.device) * scale


def _frequencies(case):
    """float64 radians per token of each pair: base 10000 over the rotated part; for a stretched context the pairs that
    turn less than once in 4096 tokens are slowed by the factor, those that turn 32 times or more are kept."""
    rot, factor = case["rot"], case["factor"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor == 1.0:
        return f, 1.0
    keep = ((4096.0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed + 1)
    op, b, page = case["op"], case["batch"], case["page"]
    new, past = _lengths(case)
    total = int(new.sum())
    s = {"case": case, "op": op, "total": total, "indptr": _indptr(new).to(dev)}
    need = 256
    if op == "pages":
        # tables that still hold pages behind the lengths (tokens cut since); the pool has room for the new ones
        cut = torch.arange(b, dtype=torch.int32) * 7 % (4 * page + 1)
        spare = int(((past + new + page - 1) // page).sum()) + 64
        table, pages = _tables(past + cut, page, cpu, spare)
        width = int(((past + torch.maximum(cut, new) + page - 1) // page).max())
        wide = torch.full((b, max(1, width)), -1, dtype=torch.int32)
        wide[:, :table.shape[1]] = table
        is_free = torch.ones((pages + 31) // 32 * 32, dtype=torch.int64)
        is_free[pages:] = 0
        is_free[table[table >= 0].long()] = 0
        words = (is_free.reshape(-1, 32) << torch.arange(32)).sum(1)
        words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
        s.update(table=wide.to(dev), lens=past.to(dev), free=words.to(dev), pages=pages)
    elif op == "rope":
        hkv, hq = case["hkv"], case["hkv"] * case["g"]
        table, pages = _tables(past + new, page, cpu, 3)
        req = torch.repeat_interleave(torch.arange(b), new.long())
        at = past[req].long() + torch.arange(total) - _indptr(new)[req].long()
        s["positions"] = at.to(torch.int32).to(dev)
        s["slots"] = (table[req, at // page].long() * page + at % page).to(dev)
        dtype = _TORCH[case["dtype"]]
        # one projection's output: queries, keys and values side by side
        qkv = _normal((total, hq + 2 * hkv, D), gen).to(dtype)
        channel = torch.exp(0.5 * _normal((hkv, D), gen))
        qkv[:, hq:hq + hkv] = (qkv[:, hq:hq + hkv].float() * channel).to(dtype)
        s.update(q=qkv[:, :hq], k_new=qkv[:, hq:hq + hkv], v_new=qkv[:, hq + hkv:])
        f, s["amp"] = _frequencies(case)
        s["freq"] = f.to(dev)
        s["k_scale"], s["v_scale"] = (0.5, 0.0625) if case["kind"] == "e4m3" else (1.0, 1.0)
        for n in ("k", "v"):
            pool = torch.zeros((pages, page, hkv, D), dtype=torch.uint8 if case["kind"] == "e4m3" else _TORCH[case["kind"]], device=dev)
            s[n] = pool
    else:
        hkv = case["hkv"]
        dtype = _TORCH[case["dtype"]]
        table, pages = _tables(past + new, page, cpu, 3)
        channel = torch.exp(0.5 * _normal((hkv, D), gen))
        s["k"] = (_normal((pages, page, hkv, D), gen) * channel).to(dtype)
        s["v"] = _normal((pages, page, hkv, D), gen).to(dtype)
        s["q"] = (_normal((total, hkv * case["g"], D), gen) * torch.exp(0.5 * _normal((total, 1, 1), gen))).to(dtype)
        s.update(table=table.to(dev), lens=(past + new).to(dev), scale=1.0 / math.sqrt(D))
    if own:
        import paged_kv_cascade_gb300 as pkc
        s["ws"] = torch.empty(pkc.chunk_workspace_size() if op == "chunk" else need, dtype=torch.uint8, device=dev)
        pkc.workspace_init(s["ws"])
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _owner(s):
    """Request of every new token."""
    row = torch.arange(s["total"], device=s["indptr"].device)
    return row, torch.searchsorted(s["indptr"], row.int(), right=True) - 1


def _pages_plain(s):
    table, lens, free, page = s["table"], s["lens"].long(), s["free"], s["case"]["page"]
    pages, dev = s["pages"], s["table"].device
    bit = torch.arange(32, device=dev)
    is_free = torch.zeros(free.numel() * 32 + 1, dtype=torch.int64, device=dev)
    is_free[:-1] = ((free[:, None] >> bit) & 1).reshape(-1)
    have = (lens + page - 1) // page
    column = torch.arange(table.shape[1], device=dev)
    # give back
    behind = (column >= have[:, None]) & (table >= 0)
    is_free[torch.where(behind, table.long(), torch.full_like(table, free.numel() * 32, dtype=torch.int64))] = 1
    held = torch.where(behind, torch.full_like(table, -1), table)
    # take: the free pages by rank
    flags = is_free[:pages]
    rank = torch.cumsum(flags, 0) - 1
    by_rank = torch.zeros(pages + 1, dtype=torch.int64, device=dev)
    by_rank[torch.where(flags > 0, rank, torch.full_like(rank, pages))] = torch.arange(pages, device=dev)
    new = (s["indptr"][1:] - s["indptr"][:-1]).long()
    need = (lens + new + page - 1) // page - have
    off = torch.cumsum(need, 0) - need
    served = off + need <= flags.sum()
    j = column - have[:, None]
    mine = (j >= 0) & (j < need[:, None]) & served[:, None]
    ranks = (off[:, None] + j).clamp(0, pages - 1)
    held = torch.where(mine, by_rank[ranks].to(torch.int32), held)
    taken = torch.where(served, need, torch.zeros_like(need)).sum()
    left = flags * (rank >= taken)
    left = torch.cat((left, torch.zeros(free.numel() * 32 - pages, dtype=torch.int64, device=dev)))
    words = (left.reshape(-1, 32) << bit).sum(1)
    free.copy_(torch.where(words >= 1 << 31, words - (1 << 32), words))
    table.copy_(held)
    # where the tokens go
    row, req = _owner(s)
    at = lens[req] + row - s["indptr"][req].long()
    entry = held[req, (at // page).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(served[req], entry * page + at % page, torch.full_like(at, -1))
    after = torch.where(served, lens + new, lens).to(torch.int32)
    return {"table": table, "free": free, "slots": slots, "positions": at.to(torch.int32), "lens": after}


def _turned(x, cos, sin, case):
    """float32 x [T, H, 128] with its first `rot` elements turned; cos, sin [T, 1, rot / 2]."""
    rot = case["rot"]
    part = x[..., :rot]
    if case["inter"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).reshape(part.shape)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((part, x[..., rot:]), -1)


def _rope_plain(s):
    case = s["case"]
    angle = s["positions"].double()[:, None, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["amp"]).float(), (torch.sin(angle) * s["amp"]).float()
    q = _turned(s["q"].float(), cos, sin, case).to(s["q"].dtype)
    k = _turned(s["k_new"].float(), cos, sin, case)
    out = []
    for n, rows in (("k", k), ("v", s["v_new"].float())):
        pool = s[n]
        flat = pool.view(-1, *pool.shape[2:])
        if pool.dtype == torch.uint8:
            rows = (rows / s[n + "_scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        flat[s["slots"]] = rows.to(pool.dtype)
        out.append(pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool)
    return {"q": q, "k": out[0], "v": out[1]}


def _tokens(pool, table):
    """A pool's rows in request order: float32 [B, Hkv, pages * page, 128] (unused pages read as page 0)."""
    x = pool[table.clamp(min=0).long()]
    return x.reshape((x.shape[0], x.shape[1] * x.shape[2]) + x.shape[3:]).permute(0, 2, 1, 3).float()


def _chunk_plain(s):
    case, indptr, lens = s["case"], s["indptr"].long(), s["lens"].long()
    b, hkv, g, dev = case["batch"], case["hkv"], case["g"], s["q"].device
    k = _tokens(s["k"], s["table"])
    t = k.shape[2]
    most = min(case["new_hi"], s["total"])
    i = torch.arange(most, device=dev)
    n = indptr[1:] - indptr[:-1]
    rows = s["q"].float()[(indptr[:-1, None] + i).clamp(max=s["total"] - 1)]  # [B, most, Hq, 128]
    q = rows.reshape(b, most, hkv, g, D).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * most, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).reshape(b, hkv, g, most, t)
    at = lens[:, None] - n[:, None] + i  # [B, most]
    token = torch.arange(t, device=dev)
    seen = (token <= at[..., None]) & (token < lens[:, None, None])
    if case["window"]:
        seen &= token > at[..., None] - case["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    o = torch.matmul(p.reshape(b, hkv, g * most, t), _tokens(s["v"], s["table"])).reshape(b, hkv, g, most, D)
    o = o / total.clamp(min=1e-38)
    row, req = _owner(s)
    j = row - indptr[req]
    o = o.permute(0, 3, 1, 2, 4)[req, j].reshape(s["q"].shape)
    lse = lse.permute(0, 3, 1, 2)[req, j].reshape(s["q"].shape[:2])
    return {"o": o.to(s["q"].dtype), "lse": lse}


def run(s):
    op, case = s["op"], s["case"]
    if not own:
        return {"pages": _pages_plain, "rope": _rope_plain, "chunk": _chunk_plain}[op](s)
    import paged_kv_cascade_gb300 as pkc
    if op == "pages":
        pkc.release_pages(s["table"], s["lens"], s["free"], case["page"], s["pages"], s["ws"])
        slots, positions, lens = pkc.assign_pages(s["table"], s["lens"], s["indptr"], s["total"], s["free"], case["page"], s["pages"], s["ws"])
        return {"table": s["table"], "free": s["free"], "slots": slots, "positions": positions, "lens": lens}
    if op == "rope":
        q = pkc.rope_append_kv(s["q"], s["k_new"], s["v_new"], s["positions"], s["slots"], s["freq"], s["k"], s["v"], s["ws"], interleaved=case["inter"],
                               amplitude=s["amp"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        k, v = ((x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x) for x in (s["k"], s["v"]))
        return {"q": q, "k": k, "v": v}
    o, lse = pkc.paged_chunk_state(s["q"], s["indptr"], s["k"], s["v"], s["table"], s["lens"], s["scale"], s["ws"], window=case["window"])
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------

def _reach(case):
    """(keys attended by all rows, cached tokens in the reach of any row), summed over the requests."""
    new, past = (x.double() for x in _lengths(case))
    w, both = case["window"], new + past
    if not w:
        return float((new * past + new * (new + 1) / 2).sum()), float(both.sum())
    short = (w - past).clamp(min=0).minimum(new)  # rows whose window still starts at the first token
    keys = short * past + short * (short + 1) / 2 + (new - short) * w
    return float(keys.sum()), float(torch.minimum(both, new + (w - 1)).sum())


def work(case):
    """Bytes: each input read once, each output written once."""
    op, page = case["op"], case["page"]
    new, past = (x.double() for x in _lengths(case))
    n, b = float(new.sum()), case["batch"]
    if op == "pages":
        fresh = float((((past + new) / page).ceil() - (past / page).ceil()).sum())
        cut = 2.0 * b  # pages given back: about two a request
        return {"bytes": 12 * n + 4 * (fresh + 2 * cut + 3 * b) + 2 * float(((past + new) / page).ceil().sum()) / 8, "flops": n}
    hq = case["hkv"] * case["g"]
    if op == "rope":
        row = 128 if case["kind"] == "e4m3" else 256
        return {"bytes": n * (512 * hq + 2 * case["hkv"] * (256 + row) + 12), "flops": 3.0 * n * (hq + case["hkv"]) * case["rot"]}
    keys, reach = _reach(case)
    return {"bytes": n * hq * (4 * D + 4) + reach * case["hkv"] * 4 * D + 4 * reach / page, "flops": 4.0 * D * hq * keys}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _nearest_e4m3(x):
    """float64 values of e4m3 nearest to x: 3 mantissa bits, exponents from -6 up, steps of 2^-9 below, at most 448."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.pow(2.0, e - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), x)


def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "rope":
        rot, out = case["rot"], {}
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None, None] * s["freq"]) * s["amp"]
        for n in ("q", "k_new"):
            x = s[n].double()
            first = torch.arange(rot // 2, device="cuda") * (2 if case["inter"] else 1)
            second = first + (1 if case["inter"] else rot // 2)
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            out[n] = x
        got = {"q": out["q"]}
        for n, rows in (("k", out["k_new"]), ("v", s["v_new"].double())):
            pool = torch.zeros(s[n].shape, dtype=torch.float64, device="cuda")
            if case["kind"] == "e4m3":
                rows = _nearest_e4m3(rows / s[n + "_scale"])
            pool.view(-1, *pool.shape[2:])[s["slots"]] = rows
            got[n] = pool
        return got
    hkv, g, page = case["hkv"], case["g"], case["page"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    ends, lens = s["indptr"].tolist(), s["lens"].tolist()
    for b, length in enumerate(lens):
        lo, hi = ends[b], ends[b + 1]
        if lo == hi:
            continue
        pages = s["table"][b, :(length + page - 1) // page].long()
        at = torch.arange(length - (hi - lo), length, device="cuda")[:, None]
        token = torch.arange(length, device="cuda")
        out = (token > at) | (token <= at - case["window"]) if case["window"] else token > at
        for h in range(hkv):
            k, v = (s[n][pages, :, h].flatten(0, 1)[:length].double() for n in ("k", "v"))
            x = torch.einsum("nhd,td->hnt", s["q"][lo:hi, h * g:(h + 1) * g].double(), k) * s["scale"]
            x.masked_fill_(out, -math.inf)
            part = torch.logsumexp(x, -1)
            lse[lo:hi, h * g:(h + 1) * g] = part.T
            o[lo:hi, h * g:(h + 1) * g] = torch.einsum("hnt,td->nhd", torch.exp(x - part[..., None]), v)
    return {"o": o, "lse": lse}
