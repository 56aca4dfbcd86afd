"""Cases of the compressed, bounded KV cache: the microscaled 4-bit (mx4) paged
cache -- quantising append, read-back, decode attention -- and eviction from a
paged cache by accumulated attention weight: accumulate, select, compact.

`run` computes each operator in elementary torch operations (32-bit), or, with
`own` set, through the library's calls.  `exact` computes the same outputs from
the definitions in 64 bits.

The mx4 format.  A head's 128 values of one token are 64 bytes of codes and 4
scale bytes.  Block b (values 32 b .. 32 b + 31) has scale byte s_b, standing
for 2^(s_b - 127) (255: NaN); a code is sign, 2 exponent bits, 1 mantissa bit
(0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).  Value 32 b + 4 u + i is
nibble i of the 16-bit little-endian word 4 u + b.
"""
import math

import torch

own = False

D = 128
PAGE = 16  # the page size of the repository's workloads

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decode step's new tokens, a serving batch: latency
        {"name": "append_step", "op": "append", "batch": 64, "hkv": 8, "lo": 1, "hi": 1, "page": PAGE, "dtype": "bf16"},
        # ragged prompts entering the cache
        {"name": "append_prompts", "op": "append", "batch": 24, "hkv": 8, "lo": 1, "hi": 8192, "page": PAGE, "dtype": "f16"},
        # a small interactive batch, one query head per KV head, no plan: latency
        {"name": "decode_tiny", "op": "decode", "batch": 4, "hkv": 32, "g": 1, "lens": "uniform", "lo": 32, "hi": 300, "page": PAGE, "dtype": "f16", "ctas": 0},
        # the GQA serving batch of the benchmark (32 / 8 heads, lognormal lengths), planned
        {"name": "decode_gqa", "op": "decode", "batch": 256, "hkv": 8, "g": 4, "lens": "lognormal", "lo": 16, "hi": 8192, "page": PAGE, "dtype": "f16", "ctas": 304},
        # two long documents: the work is split over the cache's length
        {"name": "decode_long", "op": "decode", "batch": 2, "hkv": 4, "g": 8, "lens": "uniform", "lo": 100001, "hi": 131072, "page": PAGE, "dtype": "bf16", "ctas": 304},
        # weights of a small batch's step over a 16-bit cache: latency
        {"name": "weights_tiny", "op": "weights", "batch": 4, "hkv": 32, "g": 1, "lens": "uniform", "lo": 32, "hi": 300, "page": PAGE, "kind": "f16"},
        # weights of a serving batch over a bf16 cache
        {"name": "weights_bf16", "op": "weights", "batch": 64, "hkv": 8, "g": 4, "lens": "uniform", "lo": 512, "hi": 4096, "page": PAGE, "kind": "bf16"},
        # the benchmark's GQA lengths over an mx4 cache
        {"name": "weights_mx4", "op": "weights", "batch": 256, "hkv": 8, "g": 4, "lens": "lognormal", "lo": 16, "hi": 8192, "page": PAGE, "kind": "mx4"},
        # a serving batch whose caches are cut to a budget
        {"name": "select_batch", "op": "select", "batch": 64, "hkv": 8, "lo": 1024, "hi": 16384, "budget": 1024, "sinks": 4, "recent": 256},
        # one long document: few rows, long ones
        {"name": "select_long", "op": "select", "batch": 1, "hkv": 8, "lo": 131001, "hi": 131072, "budget": 16384, "sinks": 4, "recent": 1024},
        # the cut itself, 16-bit cache
        {"name": "compact_bf16", "op": "compact", "batch": 64, "hkv": 8, "lo": 1024, "hi": 6144, "budget": 1024, "sinks": 4, "recent": 256, "page": PAGE, "kind": "bf16"},
        # a small batch over an fp8 cache, some requests within the budget: latency
        {"name": "compact_e4m3", "op": "compact", "batch": 5, "hkv": 4, "lo": 100, "hi": 777, "budget": 333, "sinks": 4, "recent": 32, "page": PAGE, "kind": "e4m3"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "decode", "weights", "weights", "select", "compact"))
    hkv = rng.choice((1, 2, 4, 8))
    page = rng.choice((8, 16, 16, 32))
    if op == "append":
        hi = _log_int(rng, 1, 8192)
        batch = _log_int(rng, 1, max(1, min(200, 65536 // hi)))
        return {"op": op, "batch": batch, "hkv": hkv, "lo": 1, "hi": hi, "page": page, "dtype": rng.choice(("f16", "bf16"))}
    hi = _log_int(rng, 33, 65536)
    batch = _log_int(rng, 1, max(1, min(256, (1 << 19) // hi)))
    lo = max(1, hi // rng.choice((2, 3, 8, 50)))
    if op == "decode":
        return {"op": op, "batch": batch, "hkv": hkv, "g": rng.choice((1, 2, 4, 8)), "lens": "uniform", "lo": lo, "hi": hi, "page": page,
                "dtype": rng.choice(("f16", "bf16")), "ctas": rng.choice((148, 304)) if hi > 1000 else 0}
    if op == "weights":
        return {"op": op, "batch": batch, "hkv": hkv, "g": rng.choice((1, 2, 4, 8)), "lens": "uniform", "lo": lo, "hi": hi, "page": page,
                "kind": rng.choice(("f16", "bf16", "e4m3", "mx4"))}
    sinks = rng.randint(0, 4)
    budget = _log_int(rng, 16, max(17, hi // 2))
    case = {"op": op, "batch": batch, "hkv": hkv, "lo": lo, "hi": hi, "budget": budget, "sinks": sinks, "recent": rng.randint(1, budget - sinks)}
    if op == "compact":
        case.update(batch=max(1, min(batch, (1 << 18) // hi)), page=page, kind=rng.choice(("f16", "bf16", "e4m3")))
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def _lengths(case):
    """The requests' lengths: the case's own, so that its outputs have one shape for every seed."""
    b = case["batch"]
    gen_cpu = torch.Generator().manual_seed(12345 + b + case["hi"])
    if case.get("lens") == "lognormal":
        x = torch.exp(7.0 + torch.randn(b, generator=gen_cpu, dtype=torch.float64))
        return x.round().clamp(case["lo"], case["hi"]).to(torch.int32)
    return torch.randint(case["lo"], case["hi"] + 1, (b,), generator=gen_cpu, dtype=torch.int32)


def _tables(lens, page, gen_cpu, dev):
    """Block table [B, max pages] (-1 unused) over a permuted pool, and the pool's pages."""
    need = (lens.long() + page - 1) // page
    total, width = int(need.sum()), max(1, int(need.max()))
    perm = torch.randperm(total, generator=gen_cpu).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    mine = torch.arange(width)[None, :] < need[:, None]
    table[mine] = perm
    return table.to(dev), total


def _normal(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device=gen.device) * scale


def _pool(shape, gen, dtype, channel=None):
    """Normal values of a cache; a scale per channel where asked (keys have channels that are larger than others)."""
    x = torch.empty(shape, dtype=dtype, device=gen.device)
    step = max(1, (1 << 27) // max(1, x[0].numel()))
    for i in range(0, shape[0], step):
        y = _normal(x[i:i + step].shape, gen)
        x[i:i + step] = (y if channel is None else y * channel).to(dtype)
    return x


def _mx4_pool(shape, gen, channel=None):
    """Codes [P, page, Hkv, 64] and scales [P, page, Hkv, 4] of a cache filled with normal values."""
    codes = torch.empty(shape[:-1] + (64,), dtype=torch.uint8, device=gen.device)
    scales = torch.empty(shape[:-1] + (4,), dtype=torch.uint8, device=gen.device)
    step = max(1, (1 << 25) // max(1, shape[1] * shape[2] * D))
    for i in range(0, shape[0], step):
        y = _normal((min(step, shape[0] - i),) + shape[1:], gen)
        codes[i:i + step], scales[i:i + step] = _quantise((y if channel is None else y * channel).half().float())
    return codes, scales


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed + 1)
    op, b, hkv = case["op"], case["batch"], case["hkv"]
    s = {"case": case, "op": op, "scale": 1.0 / math.sqrt(D)}
    lens = _lengths(case)
    ctas = case.get("ctas", 0)
    if op == "append":
        n_new, old = lens, (torch.arange(b, dtype=torch.int32) * 37 + 11) % 100
        s["table"], pages = _tables(old + n_new, case["page"], cpu, dev)
        indptr = torch.zeros(b + 1, dtype=torch.int32)
        indptr[1:] = torch.cumsum(n_new, 0)
        total = int(indptr[-1])
        channel = torch.exp(0.7 * _normal((hkv, D), gen))
        s.update(k_new=_pool((total, hkv, D), gen, _TORCH[case["dtype"]], channel), v_new=_pool((total, hkv, D), gen, _TORCH[case["dtype"]]),
                 indptr=indptr.to(dev), lens=old.to(dev), total=total)
        for n in ("k", "v"):
            s[n + "_codes"] = torch.zeros((pages, case["page"], hkv, 64), dtype=torch.uint8, device=dev)
            s[n + "_scales"] = torch.zeros((pages, case["page"], hkv, 4), dtype=torch.uint8, device=dev)
    elif op in ("decode", "weights"):
        s["table"], pages = _tables(lens, case["page"], cpu, dev)
        s["lens"] = lens.to(dev)
        shape = (pages, case["page"], hkv, D)
        kind = case.get("kind", "mx4")
        channel = torch.exp(0.5 * _normal((hkv, D), gen))
        dtype = _TORCH[case["dtype"] if op == "decode" else kind if kind in _TORCH else "f16"]
        s["q"] = (_normal((b, hkv * case["g"], D), gen) * torch.exp(0.5 * _normal((b, 1, 1), gen))).to(dtype)
        s["k_scale"] = 0.5 if kind == "e4m3" else 1.0
        if kind == "mx4":
            s["k"], s["k_scales"] = _mx4_pool(shape, gen, channel)
        elif kind == "e4m3":
            s["k"] = _pool(shape, gen, torch.float8_e4m3fn, channel).view(torch.uint8)
        else:
            s["k"] = _pool(shape, gen, _TORCH[kind], channel)
        if op == "decode":
            s["v"], s["v_scales"] = _mx4_pool(shape, gen)
        else:
            width = s["table"].shape[1] * case["page"]
            s["weights"] = torch.rand((b, hkv, width), generator=gen, device=dev)
            s["lse"] = _lse_of(s)
    else:
        s["lens"] = lens.to(dev)
        width = (int(lens.max()) + 63) // 64 * 64
        # accumulated weights spread over decades; many late tokens have none yet
        w = torch.exp(3.0 * _normal((b, hkv, width), gen) - 6.0)
        s["weights"] = torch.where(torch.rand(w.shape, generator=gen, device=dev) < 0.1, torch.zeros_like(w), w)
        if op == "compact":
            s["table"], pages = _tables(lens, case["page"], cpu, dev)
            shape = (pages, case["page"], hkv, D)
            dtype = torch.float8_e4m3fn if case["kind"] == "e4m3" else _TORCH[case["kind"]]
            for n in ("k", "v"):
                x = _pool(shape, gen, dtype)
                s[n] = x.view(torch.uint8) if case["kind"] == "e4m3" else x
            s["keep"] = _select(s["weights"], s["lens"], case["budget"], case["sinks"], case["recent"])
    if own:
        import paged_kv_cascade_gb300 as pkc
        heads = hkv * case.get("g", 1)
        s["ws"] = torch.empty(pkc.workspace_size(b, heads, ctas, 0), dtype=torch.uint8, device=dev)
        pkc.workspace_init(s["ws"])
        if ctas:
            s["plan"] = pkc.plan(lens.numpy(), ctas)
            pkc.plan_upload(s["plan"], s["ws"])
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _quantise(x):
    """Codes [..., 64] and scales [..., 4] of float32 x [..., 128]."""
    y = x.reshape(x.shape[:-1] + (4, 32))
    amax = y.abs().amax(-1)
    finite = torch.isfinite(amax)
    exponent = torch.frexp(torch.where(finite, amax, torch.ones_like(amax)))[1] - 1  # floor(log2 amax)
    exponent = torch.where(amax > 0, exponent - 2, torch.full_like(exponent, -126)).clamp(min=-126)
    scales = torch.where(finite, exponent + 127, torch.full_like(exponent, 255)).to(torch.uint8)
    z = torch.ldexp(y, -exponent[..., None])
    a = z.abs()
    # nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code; above 6: 6
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8)
            + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    code = code | (torch.signbit(z).to(torch.uint8) << 3)
    code = torch.where(finite[..., None], code, torch.zeros_like(code))
    nib = code.reshape(x.shape[:-1] + (4, 8, 2, 2)).transpose(-4, -3)  # [..., u, b, byte, low / high]
    return (nib[..., 0] | (nib[..., 1] << 4)).reshape(x.shape[:-1] + (64,)), scales


_BYTES = {}


def _values(codes, scales):
    """float32 [..., 128] of codes and scales."""
    dev = codes.device
    if dev not in _BYTES:
        signed = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=dev)
        byte = torch.arange(256, device=dev)
        _BYTES[dev] = torch.stack((signed[byte % 16], signed[byte // 16]), -1)
    v = torch.index_select(_BYTES[dev], 0, codes.reshape(-1).int()).reshape(codes.shape[:-1] + (8, 4, 4)).transpose(-3, -2)
    e = torch.where(scales == 255, torch.full_like(scales, 0, dtype=torch.float32) + math.nan,
                    torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127))
    return (v * e[..., None, None]).reshape(codes.shape[:-1] + (D,))


def _tokens(pool, table):
    """A pool's rows in request order: [B, pages * page, Hkv, ...] (unused pages read as page 0)."""
    x = pool[table.clamp(min=0).long()]
    return x.reshape((x.shape[0], x.shape[1] * x.shape[2]) + x.shape[3:])


def _keys(s):
    rows = _tokens(s["k"], s["table"])
    if "k_scales" in s:
        return _values(rows, _tokens(s["k_scales"], s["table"]))
    if s["k"].dtype == torch.uint8:
        return rows.view(torch.float8_e4m3fn).float() * s["k_scale"]
    return rows.float()


def _scores(s):
    """[B, Hkv, G, T] scores; -inf past each request's end."""
    k = _keys(s)
    b, t, hkv, _ = k.shape
    q = s["q"].float().reshape(b, hkv, -1, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    past = torch.arange(t, device=x.device)[None, :] >= s["lens"][:, None]
    return x.masked_fill_(past[:, None, None, :], -math.inf)


def _softmax_parts(x):
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    return p, total, (m + torch.log(total)).squeeze(-1)


def _lse_of(s):
    return _softmax_parts(_scores(s))[2].reshape(s["q"].shape[:2])


def _select(weights, lens, budget, sinks, recent):
    """[B, Hkv, budget]: the kept slots in ascending order, -1 behind them."""
    b, hkv, width = weights.shape
    slot = torch.arange(width, device=weights.device)
    n = lens[:, None, None]
    inf = torch.full_like(weights, math.inf)
    key = torch.where(slot < sinks, inf, weights)
    key = torch.where(slot < n - recent, key, -inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1]
    top = torch.zeros_like(weights, dtype=torch.bool)
    top.scatter_(-1, order[..., :max(0, budget - recent)], True)
    kept = torch.where(n > budget, top | (slot >= n - recent), slot < n) & (slot < n)
    where = torch.where(kept, slot, torch.full_like(slot, width))
    where = torch.sort(where, dim=-1)[0][..., :budget]
    keep = torch.where(where < width, where, torch.full_like(where, -1)).to(torch.int32)
    if budget > width:
        keep = torch.cat((keep, torch.full((b, hkv, budget - width), -1, dtype=torch.int32, device=keep.device)), -1)
    return keep


def _append_plain(s, lens):
    total, indptr, page = s["total"], s["indptr"], s["case"]["page"]
    row = torch.arange(total, device=indptr.device)
    req = torch.searchsorted(indptr, row.int(), right=True) - 1
    at = lens[req].long() + row - indptr[req].long()
    pages = s["table"][req, at // page].long()
    out = []
    for n in ("k", "v"):
        codes, scales = _quantise(s[n + "_new"].float())
        s[n + "_codes"][pages, at % page] = codes
        s[n + "_scales"][pages, at % page] = scales
        out.append(_values(codes, scales).to(s[n + "_new"].dtype))
    lens += indptr[1:] - indptr[:-1]
    return {"k": out[0], "v": out[1], "lens": lens}


def _decode_plain(s):
    p, total, lse = _softmax_parts(_scores(s))
    v = _values(_tokens(s["v"], s["table"]), _tokens(s["v_scales"], s["table"]))
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / total.clamp(min=1e-38)
    return {"o": o.reshape(s["q"].shape).to(s["q"].dtype), "lse": lse.reshape(s["q"].shape[:2])}


DECAY = 0.75


def _weights_plain(s):
    b, hkv, width = s["weights"].shape
    x = torch.exp(_scores(s) - s["lse"].reshape(b, hkv, -1, 1)).sum(2)
    live = torch.arange(width, device=x.device) < s["lens"][:, None, None]
    w = s["weights"]
    w.copy_(torch.where(live, DECAY * w + x, w))
    return {"weights": w}


def _compact_plain(s, lens):
    keep, table, page = s["keep"], s["table"], s["case"]["page"]
    b, hkv, budget = keep.shape
    cut = lens > budget
    # rows that move: (request, head, new slot)
    req, head, new = torch.nonzero(cut[:, None, None].expand(b, hkv, budget), as_tuple=True)
    src = keep[req, head, new].long()
    at, to = (table[req, src // page].long(), src % page), (table[req, new // page].long(), new % page)
    for n in ("k", "v"):
        s[n][to[0], to[1], head] = s[n][at[0], at[1], head]
    w = s["weights"]
    kept = torch.gather(w, -1, keep.clamp(min=0).long())
    after = torch.zeros_like(w)
    after[..., :budget] = kept
    slot = torch.arange(w.shape[-1], device=w.device)
    w.copy_(torch.where(cut[:, None, None] & (slot < lens[:, None, None]), after, w))
    lens.clamp_(max=budget)


def run(s):
    op = s["op"]
    if own:
        import paged_kv_cascade_gb300 as pkc
    if op == "append":
        lens = s["lens"].clone()
        if not own:
            return _append_plain(s, lens)
        pools = (s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
        pkc.append_kv_mx4(s["k_new"], s["v_new"], s["indptr"], *pools, s["table"], lens, s["ws"])
        k, v = pkc.gather_kv_mx4(*pools, s["table"], s["lens"], s["indptr"], s["total"], s["ws"], dtype=s["k_new"].dtype)
        return {"k": k, "v": v, "lens": lens}
    if op == "decode":
        if not own:
            return _decode_plain(s)
        o, lse = pkc.paged_decode_state_mx4(s["q"], s["k"], s["k_scales"], s["v"], s["v_scales"], s["table"], s["lens"], s["scale"], s["ws"],
                                            plan_buf=s.get("plan"))
        return {"o": o, "lse": lse}
    if op == "weights":
        if not own:
            return _weights_plain(s)
        pkc.accumulate_weights(s["q"], s["lse"], s["k"], s["table"], s["lens"], s["scale"], s["weights"], s["ws"], decay=DECAY,
                               k_scale=s["k_scale"], k_scales=s.get("k_scales"))
        return {"weights": s["weights"]}
    case = s["case"]
    if op == "select":
        if not own:
            return {"keep": _select(s["weights"], s["lens"], case["budget"], case["sinks"], case["recent"])}
        return {"keep": pkc.evict_select(s["weights"], s["lens"], case["budget"], case["sinks"], case["recent"], s["ws"])}
    lens = s["lens"].clone()
    if own:
        pkc.evict_compact(s["keep"], s["k"], s["v"], s["table"], lens, s["ws"], weights=s["weights"])
    else:
        _compact_plain(s, lens)
    k, v = ((x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x) for x in (s["k"], s["v"]))
    return {"k": k, "v": v, "weights": s["weights"], "lens": lens}


# ---------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------

def work(case):
    """Bytes: each input read once, each output written once."""
    op, b, hkv = case["op"], case["batch"], case["hkv"]
    lens = _lengths(case).double()
    n, page = float(lens.sum()), case.get("page", PAGE)
    if op == "append":
        rows = 2.0 * n * hkv
        # 16-bit rows in, 68-byte rows out, then those rows in and 16-bit rows out
        return {"bytes": rows * (256 + 68 + 68 + 256) + 12 * b, "flops": rows * D * 4}
    if op == "decode":
        heads = hkv * case["g"]
        return {"bytes": 2 * n * hkv * 68 + b * heads * (4 * D + 4) + 4 * n / page, "flops": 4.0 * n * heads * D}
    if op == "weights":
        heads = hkv * case["g"]
        row = {"f16": 256, "bf16": 256, "e4m3": 128, "mx4": 68}[case["kind"]]
        return {"bytes": n * hkv * (row + 8) + b * heads * (2 * D + 4) + 4 * n / page, "flops": 2.0 * n * heads * D}
    kept = float(lens.clamp(max=case["budget"]).sum())
    if op == "select":
        return {"bytes": 4.0 * hkv * (n + b * case["budget"]), "flops": n * hkv}
    moved = float((lens > case["budget"]).sum()) * case["budget"]
    row = 128 if case["kind"] == "e4m3" else 256
    return {"bytes": hkv * (moved * (4 * row + 4) + 4 * kept + 4 * n), "flops": moved * hkv}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _decode_row64(codes, scales):
    """float64 [..., 128]: sign, exponent and mantissa of every nibble, by the format's definition."""
    d = torch.arange(D, device=codes.device)
    block, u, i = d // 32, d % 32 // 4, d % 4
    byte = codes[..., 2 * (4 * u + block) + i // 2].to(torch.int64)
    nib = (byte >> (4 * (i % 2))) & 15
    exp, man, sign = (nib >> 1) & 3, nib & 1, 1 - 2 * (nib >> 3)
    mag = torch.where(exp > 0, torch.pow(2.0, (exp - 1).double()) * (1 + 0.5 * man), 0.5 * man.double())
    s = scales[..., block].double()
    return torch.where(s == 255, torch.full_like(mag, math.nan), sign * mag * torch.pow(2.0, s - 127))


def _nearest64(x):
    """float64 values that quantising x [..., 128] gives: the nearest code of the block's scale, the even one of two."""
    y = x.double().reshape(x.shape[:-1] + (4, 32))
    amax = y.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -130)))
    e = torch.where(torch.pow(2.0, e) > amax, e - 1, e)  # the logarithm may round over a border, either way
    e = torch.where(torch.pow(2.0, e + 1) <= amax, e + 1, e)
    scale = torch.pow(2.0, (e - 2).clamp(min=-126))
    a = (y / scale).abs()
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    best, off = torch.zeros_like(a), a.clone()
    for code in (2, 4, 6, 1, 3, 5, 7):  # the even codes first: they keep ties
        nearer = (a - grid[code]).abs() < off
        best, off = torch.where(nearer, grid[code], best), torch.where(nearer, (a - grid[code]).abs(), off)
    return (torch.copysign(best, y) * scale).reshape(x.shape)


def _request64(s, name, b, n):
    """float64 [n, Hkv, 128] of request b's first n cached tokens."""
    pages = s["table"][b, :(n + s["case"]["page"] - 1) // s["case"]["page"]].long()
    rows = s[name][pages].flatten(0, 1)[:n]
    if name + "_scales" in s:
        return _decode_row64(rows, s[name + "_scales"][pages].flatten(0, 1)[:n])
    if rows.dtype == torch.uint8:
        return rows.view(torch.float8_e4m3fn).double() * s["k_scale"]
    return rows.double()


def exact(case, seed):
    s = prepare(case, seed)
    op, b, hkv = case["op"], case["batch"], case["hkv"]
    lens = s["lens"].tolist()
    if op == "append":
        out = {n: _nearest64(s[n + "_new"]) for n in ("k", "v")}
        out["lens"] = s["lens"] + s["indptr"].diff()
        return out
    if op in ("decode", "weights"):
        g = case["g"]
        q = s["q"].double().reshape(b, hkv, g, D)
        o = torch.zeros(b, hkv, g, D, dtype=torch.float64, device="cuda")
        lse = torch.full((b, hkv, g), -math.inf, dtype=torch.float64, device="cuda")
        w = s["weights"].double() if op == "weights" else None
        for i, n in enumerate(lens):
            if n == 0:
                continue
            x = torch.einsum("hgd,thd->hgt", q[i], _request64(s, "k", i, n)) * s["scale"]
            if op == "weights":
                p = torch.exp(x - s["lse"][i].double().reshape(hkv, g, 1))
                w[i, :, :n] = DECAY * w[i, :, :n] + p.sum(1)
            else:
                lse[i] = torch.logsumexp(x, -1)
                o[i] = torch.einsum("hgt,thd->hgd", torch.exp(x - lse[i][..., None]), _request64(s, "v", i, n))
        if op == "weights":
            return {"weights": w}
        return {"o": o.reshape(b, hkv * g, D), "lse": lse.reshape(b, hkv * g)}
    if op == "select":
        return None  # whole numbers
    # compact: every kept row at its new place, rows of other places as they were
    out = {}
    for n in ("k", "v"):
        x = s[n].view(torch.float8_e4m3fn) if s[n].dtype == torch.uint8 else s[n]
        x = x.double()
        for i, length in enumerate(lens):
            if length > case["budget"]:
                pages = s["table"][i].clamp(min=0).long()
                rows = x[pages].flatten(0, 1)  # a copy in request order
                pick = s["keep"][i].long()
                moved = torch.stack([rows[pick[h], h] for h in range(hkv)], 1)
                rows[:case["budget"]] = moved
                used = (length + case["page"] - 1) // case["page"]
                x[pages[:used]] = rows.reshape((len(pages), case["page"]) + rows.shape[1:])[:used]
        out[n] = x
    w = s["weights"].double()
    for i, length in enumerate(lens):
        if length > case["budget"]:
            kept = torch.gather(w[i], -1, s["keep"][i].long())
            w[i, :, :length] = 0
            w[i, :, :case["budget"]] = kept
    out["weights"] = w
    out["lens"] = s["lens"].clamp(max=case["budget"])
    return out
