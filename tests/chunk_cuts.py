"""Which blocks work on which KV tiles of a chunk call's items, one item after another:
the cut that every block works out for itself in closed form."""

ROWS, TILE, SHORT = 256, 128, 12
TILE_COST, HALF_TILE_COST, ITEM_COST, LEAST_SHARE = 5, 4, 12, 16


def reach(n, length, j0, j1, causal, window):
    """KV tiles [lo, hi) of a request's new tokens j0 .. j1 - 1."""
    at = length - n
    end = at + j1 if causal else length
    begin = at + j0 - window + 1 if window else 0
    hi = -(-max(end, 0) // TILE)
    return min(max(begin, 0) // TILE, hi), hi


def pieces(reqs, hkv, g, blocks, causal=True, window=0):
    """Per item of requests (new, past): (half A's tiles, half B's tiles, [(block, first tile, end)])."""
    tokens, items, total = ROWS // g, [], 0
    for n, past in reqs:
        for _ in range(hkv):
            for j0 in range(0, n, tokens):
                j1, mid = min(n, j0 + tokens), j0 + tokens // 2
                a = reach(n, n + past, j0, min(j1, mid), causal, window)
                b = reach(n, n + past, mid, j1, causal, window) if j1 > mid else (a[1], a[1])
                cost = HALF_TILE_COST if (n - j0) * g <= ROWS // 2 else TILE_COST
                lo, hi = a[0], max(a[1], b[1])
                items.append((a, b, lo, hi, cost, total + ITEM_COST))
                total += ITEM_COST + (hi - lo) * cost
    blocks = max(1, min(blocks, total // LEAST_SHARE))
    ends = [(c + 1) * total // blocks for c in range(blocks)]
    out = []
    for a, b, lo, hi, cost, first in items:
        of = []
        for t in range(lo, hi):
            last = first + (t - lo + 1) * cost - 1 if hi - lo > SHORT else first + (hi - lo) * cost - 1
            c = next(i for i, e in enumerate(ends) if last < e)
            if of and of[-1][0] == c:
                of[-1][2] = t + 1
            else:
                of.append([c, t, t + 1])
        out.append((a, b, of))
    return out


# name: (requests of (new, past) tokens, query heads, KV heads, causal, window)
CASES = {
    "five words": ([(5, 40000)], 8, 1, True, 0),
    "several items": ([(5, 20000), (3, 15000)], 4, 2, True, 0),
    "both halves": ([(300, 6000)], 1, 1, True, 0),
    "eight heads": ([(40, 6000)], 8, 1, True, 0),
    "window": ([(300, 6000)], 1, 1, True, 3000),
    "window of eight heads": ([(40, 6000)], 8, 1, True, 3000),
    "not causal": ([(150, 5000)], 2, 1, False, 0),
    "not causal, window": ([(150, 5000)], 2, 1, False, 2500),
    "beside others": ([(1, 2500 + 37 * i) for i in range(30)] + [(70, 3000), (0, 50), (2, 10)], 4, 1, True, 0),
    "a half alone": ([(256, 3000)], 1, 1, True, 2500),
}
