"""Plain definitions, in 64 bits, of a prompt's way into the paged cache: pages
and slots, rotary positions, attention of a chunk over the cache."""
import math

import numpy as np
import torch

# half a step of each type, relative to the value
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


# ------------------------------------------------------------------- pages

def pool_words(free, num_pages):
    """The map of a set of free pages, as int32 words."""
    words = np.zeros((num_pages + 31) // 32, np.uint32)
    for p in free:
        words[p // 32] |= np.uint32(1 << (p % 32))
    return torch.from_numpy(words.view(np.int32).copy())


def pool_set(words, num_pages):
    w = words.cpu().numpy().view(np.uint32)
    return {p for p in range(num_pages) if w[p // 32] >> (p % 32) & 1}


def release(table, lens, free, page):
    """table (list of lists) and free (set) changed in place."""
    for row, n in zip(table, lens):
        for j in range(-(-n // page), len(row)):
            if row[j] >= 0:
                free.add(row[j])
                row[j] = -1


def assign(table, lens, indptr, total, free, page):
    """(slots, positions, lens out, status); table and free changed in place."""
    slots, positions, out, status = [-1] * total, [0] * total, list(lens), 0
    if any(indptr[b + 1] > indptr[b] and -(-(n + indptr[b + 1] - indptr[b]) // page) > len(table[b]) for b, n in enumerate(lens)):
        status = 4  # seen before the pages are counted
    order = sorted(free)
    at = 0  # pages counted so far, served or not
    for b, n in enumerate(lens):
        new = indptr[b + 1] - indptr[b]
        have, want = -(-n // page), -(-(n + new) // page)
        for i in range(new):
            positions[indptr[b] + i] = n + i
        if new and want > len(table[b]):
            continue
        at += want - have
        if want > have and at > len(order):
            status = status or 8
            continue
        for j in range(have, want):
            table[b][j] = order[at - (want - have) + j - have]
            free.discard(table[b][j])
        out[b] = n + new
        for i in range(new):
            slots[indptr[b] + i] = table[b][(n + i) // page] * page + (n + i) % page
    return slots, positions, out, status


# ------------------------------------------------------------------ rotary

def rotate(x, positions, inv_freq, interleaved, amplitude):
    """float64 x [T, H, 128] turned, and the sum of magnitudes that each element is made of."""
    x = x.double()
    r = 2 * len(inv_freq)
    a = positions.double()[:, None, None] * inv_freq.double()
    c, s = torch.cos(a) * amplitude, torch.sin(a) * amplitude
    i = torch.arange(r // 2)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    u, v = x[..., first], x[..., second]
    out, size = x.clone(), x.abs()
    out[..., first], out[..., second] = u * c - v * s, u * s + v * c
    size[..., first] = size[..., second] = abs(amplitude) * (u.abs() + v.abs())
    return out, size


# ------------------------------------------------------------------- chunk

def chunk(q, q_indptr, k_cache, v_cache, table, lens, scale, causal=True, window=0):
    """float64 (o, lse, and per element or row the allowed errors of a float32
    computation whose probabilities are rounded to q's type).

    With w the weights, S the largest scale * sum |q k| of a row: a score is off
    by at most 128 half-steps of float32 of its own terms and the exponent's
    argument and the exponential by a few more, d = 2^-17 S + 2^-19 together; a
    weight is then off by a share of 2 d, and by half a step of its type where
    it enters the V product (fp16: at least 2^-25 of the largest)."""
    T, hq, D = q.shape
    page, hkv = k_cache.shape[1], k_cache.shape[2]
    g = hq // hkv
    half = HALF_STEP[q.dtype]
    o = torch.zeros(T, hq, D, dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    o_tol, lse_tol = torch.zeros_like(o), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        lo, hi = q_indptr[b], q_indptr[b + 1]
        if hi == lo:
            continue
        pages = table[b][:-(-n // page)].long()
        k = k_cache[pages].reshape(-1, hkv, D)[:n].double()
        v = v_cache[pages].reshape(-1, hkv, D)[:n].double()
        at = torch.arange(n - (hi - lo), n)
        t = torch.arange(n)
        seen = torch.ones(hi - lo, n, dtype=torch.bool)
        if causal:
            seen &= t <= at[:, None]
        if window:
            seen &= t > at[:, None] - window
        for h in range(hq):
            qh, kh, vh = q[lo:hi, h].double(), k[:, h // g], v[:, h // g]
            for i in range(hi - lo):
                m = seen[i]
                if not m.any():
                    continue
                x = kh[m] @ qh[i] * scale
                size = float((kh[m].abs() @ qh[i].abs()).max() * scale)
                lse[lo + i, h] = torch.logsumexp(x, 0)
                w = torch.softmax(x, 0)  # (64 bits of x - lse are not enough where x passes 2^50)
                o[lo + i, h] = w @ vh[m]
                d = 2.0 ** -17 * size + 2.0 ** -19
                spread = w @ vh[m].abs()
                o_tol[lo + i, h] = (2 * d + half) * spread
                if q.dtype == torch.float16:
                    o_tol[lo + i, h] += 2.0 ** -25 * vh[m].abs().sum(0)
                lse_tol[lo + i, h] = d
    return o, lse, o_tol, lse_tol


def check_chunk(got_o, got_lse, want, dtype, rows=None):
    o, lse, o_tol, lse_tol = want
    go, gl = got_o.double().cpu(), got_lse.double().cpu()
    if rows is not None:
        go, gl, o, lse, o_tol, lse_tol = (x[rows] for x in (go, gl, o, lse, o_tol, lse_tol))
    empty = torch.isneginf(lse)
    assert torch.equal(torch.isneginf(gl), empty)
    assert torch.all(go[empty] == 0)
    assert torch.isfinite(go).all()
    off = (go - o).abs() - (o_tol + HALF_STEP[dtype] * (o.abs() + o_tol) + 2.0 ** -25)
    assert float(off.max()) <= 0 if off.numel() else True, f"O off by {float((go - o).abs().max()):.3e}, {float(off.max()):.3e} too far"
    far = (gl - lse).abs()[~empty] - lse_tol[~empty] - 2.0 ** -23 * lse.abs()[~empty]
    assert far.numel() == 0 or float(far.max()) <= 0, f"LSE {float(far.max()):.3e} too far"
