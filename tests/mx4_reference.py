"""The mx4 format and attention over it in float64, in numpy alone: the plain
implementation that the GPU kernels' tests compare with.

A row of 128 elements has 4 blocks of 32 with scale bytes s (2^(s - 127), 255
NaN) and 64 bytes of codes; element 32 b + 4 u + i is nibble i of the 16-bit
little-endian word 4 u + b; a nibble is sign, 2 exponent bits, 1 mantissa bit.
"""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise(x):
    """float64 x [..., 128] -> codes uint8 [..., 64], scales uint8 [..., 4]."""
    x = np.asarray(x, np.float64)
    y = x.reshape(x.shape[:-1] + (4, 32))
    with np.errstate(invalid="ignore"):
        amax = np.max(np.abs(y), axis=-1)
    finite = np.isfinite(amax)
    e = np.where(finite & (amax > 0), np.frexp(np.where(finite, amax, 1.0))[1] - 1 - 2, -126)
    e = np.maximum(e, -126)
    z = np.ldexp(np.where(finite[..., None], y, 0.0), -e[..., None])
    a = np.abs(z)
    off = np.abs(a[..., None] - GRID)
    # nearest; of two equally near ones the even code
    best = np.argmin(off + 1e-12 * (np.arange(8) % 2), axis=-1)
    code = (best | (np.signbit(z) << 3)).astype(np.uint16)
    code = np.where(finite[..., None], code, 0).astype(np.uint16)
    nib = np.swapaxes(code.reshape(x.shape[:-1] + (4, 8, 4)), -3, -2)  # [..., u, b, i]
    words = nib[..., 0] | (nib[..., 1] << 4) | (nib[..., 2] << 8) | (nib[..., 3] << 12)
    codes = np.ascontiguousarray(words.reshape(x.shape[:-1] + (32,)).astype("<u2")).view(np.uint8)
    return codes, np.where(finite, e + 127, 255).astype(np.uint8)


def values(codes, scales):
    """float64 [..., 128] of codes [..., 64] and scales [..., 4]."""
    words = np.ascontiguousarray(codes).view("<u2").reshape(codes.shape[:-1] + (8, 4))  # [..., u, b]
    nib = np.stack([(words >> (4 * i)) & 15 for i in range(4)], -1)
    v = np.where(nib & 8, -GRID[nib & 7], GRID[nib & 7])
    v = np.swapaxes(v, -3, -2).reshape(codes.shape[:-1] + (4, 32))
    s = scales.astype(np.float64)
    f = np.where(scales == 255, np.nan, np.exp2(s - 127))
    return (v * f[..., None]).reshape(codes.shape[:-1] + (128,))


def request_rows(pool, table_row, n, page_size):
    """pool [P, page_size, ...] -> the first n tokens of a request."""
    if n == 0:
        return pool[:0, 0]
    pages = table_row[:(n + page_size - 1) // page_size]
    return pool[pages].reshape((-1,) + pool.shape[2:])[:n]


def attention(q, k, v, g, scale):
    """One request in float64: q [Hq, 128], k / v [n, Hkv, 128] -> O, LSE and
    the sizes that error bounds need: per head the largest scale * sum |q k|,
    and per (head, dim) the largest |v| of the dim's block of 32."""
    hq, n, hkv = q.shape[0], k.shape[0], k.shape[1]
    o, lse = np.zeros((hq, 128)), np.full(hq, -np.inf)
    s_mag, v_mag = np.zeros(hq), np.zeros((hq, 128))
    for h in range(hq if n else 0):
        kk, vv = k[:, h // g], v[:, h // g]
        with np.errstate(invalid="ignore", over="ignore"):
            s = scale * (kk @ q[h])
            m = np.max(s)
            if not np.isfinite(m):
                m = 0.0
            p = np.exp(s - m)
            tot = p.sum()
            lse[h] = m + np.log(tot)
            o[h] = (p / tot) @ vv
            s_mag[h] = np.max(scale * (np.abs(kk) @ np.abs(q[h])))
            v_mag[h] = np.repeat(np.max(np.abs(vv).reshape(n, 4, 32), axis=(0, 2)), 32)
    return o, lse, s_mag, v_mag


def bounds(o, lse, s_mag, v_mag, eps):
    """Error bounds of a kernel's O and LSE.

    A score is a float32 sum of 128 products and a few more roundings: at most
    136 half-steps (2^-24) of scale * sum |q k|, and its conversion to base 2
    one more of |s| (also within s_mag).  A probability is off by that factor
    in its exponent, by 2^-21 for the exponential and by 2^-21 for its two-part
    16-bit form; both numerator and denominator carry it, and the weighted
    values are bounded by the block's largest |v|.  Their float32 sums add
    2^-18 of it (64 roundings of accumulation).  The result is rounded once to
    its type (eps / 2), denormals by half the smallest step.
    """
    dp = 137 * 2.0 ** -24 * s_mag + 2.0 ** -20
    o_tol = (2 * dp + 2.0 ** -18)[:, None] * v_mag + np.abs(o) * eps / 2 + 2.0 ** -25
    lse_tol = dp + 2.0 ** -18 + np.where(np.isfinite(lse), np.abs(lse), 0.0) * 2.0 ** -22
    return o_tol, lse_tol
