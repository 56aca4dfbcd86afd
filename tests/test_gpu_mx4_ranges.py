"""The mx4 cache's decode and weights at the ends of the number ranges: queries
and keys far from 1, scores beyond 2^24, values near the smallest and the
largest numbers, every scale byte."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
import paged_kv_cascade_gb300 as pkc
from test_gpu_evict import want_weights
from test_gpu_mx4 import DT, Cache, check_decode, f64, ws_for

pytestmark = pytest.mark.gpu


def want_w_of_decode(c, q, lse, w, g, scale):
    """The weights of one step against float64 ones (want_weights reads a Paged's `rows`)."""
    class View:
        lens, hkv = c.lens, c.hkv

        @staticmethod
        def rows(i, b, n):
            return (c.k, c.v)[i][b]
    want, tol = want_weights(View, q, lse, scale, np.zeros(tuple(w.shape)), 0.0, g)
    got = f64(w)
    assert np.all(np.abs(got - want) <= tol), np.nanmax(np.abs(got - want) - tol)


# ---------------------------------------------------------------------------
# Scale bytes
# ---------------------------------------------------------------------------

def smallest(c, j, rng):
    """Fill K (j 0) or V (j 2) of request 0 with any codes under scale bytes 0, 1 and 2."""
    pages = c.bt[0, :(c.lens[0] + c.ps - 1) // c.ps]
    n = len(pages) * c.ps
    codes = rng.integers(0, 256, (n, c.hkv, 64)).astype(np.uint8)
    scales = np.where(rng.random((n, c.hkv, 4)) < 0.5, 0, rng.integers(0, 3, (n, c.hkv, 4))).astype(np.uint8)
    c.pools[j][pages], c.pools[j + 1][pages] = codes.reshape(-1, c.ps, c.hkv, 64), scales.reshape(-1, c.ps, c.hkv, 4)
    (c.k, c.v)[j // 2][0] = ref.values(codes, scales)[:c.lens[0]]


@pytest.mark.parametrize("ps", [16, 5])
def test_keys_of_scale_byte_0(ps):
    """Pools that the caller filled: scale byte 0 stands for 2^-127, in the
    decode's scores and in the weights'."""
    rng = np.random.default_rng(6)
    c = Cache([70], 2, ps, rng)
    smallest(c, 0, rng)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((1, 4, 128)) * 2.0 ** 123).cuda().bfloat16()
    ws = ws_for(1, 4)
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.5, ws)
    check_decode(c, q, o, lse, 2, 0.5, "bf16")
    w = torch.zeros(1, 2, 80, device="cuda")
    pkc.accumulate_weights(q, lse, d[0], bt, dl, 0.5, w, ws, k_scales=d[1])
    want_w_of_decode(c, q, lse, w, 2, 0.5)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("ps", [16, 5])
def test_scale_byte_255_is_nan_whatever_the_codes(ps, dtype):
    """One key block (request 0) and one value block (request 1) of NaN whose
    codes are not zero."""
    rng = np.random.default_rng(7)
    c = Cache([40, 40, 40], 1, ps, rng)
    c.pools[1][c.bt[0, 7 // ps], 7 % ps, 0, 2] = 255
    c.pools[3][c.bt[1, 9 // ps], 9 % ps, 0, 1] = 255
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((3, 2, 128))).cuda().to(DT[dtype])
    ws = ws_for(3, 2)
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws)
    want_o, want_l = np.zeros((3, 2, 128), bool), np.zeros((3, 2), bool)
    want_o[0], want_l[0], want_o[1, :, 32:64] = True, True, True
    np.testing.assert_array_equal(np.isnan(f64(o)), want_o)
    np.testing.assert_array_equal(np.isnan(f64(lse)), want_l)
    w = torch.zeros(3, 1, 48, device="cuda")
    pkc.accumulate_weights(q, torch.zeros(3, 2, device="cuda"), d[0], bt, dl, 0.1, w, ws, k_scales=d[1])
    want_w = np.zeros((3, 1, 48), bool)
    want_w[0, 0, 7] = True
    np.testing.assert_array_equal(np.isnan(f64(w)), want_w)


# ---------------------------------------------------------------------------
# bf16 queries and keys whose sizes are far from 1 and cancel in the scores
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("g", [2, 8])
@pytest.mark.parametrize("power", [-120, -112, -108, -70, -50, 50, 63, 64, 65, 66, 108, 112, 118])
def test_decode_where_queries_and_keys_cancel(power, g):
    """|q| about 2^power, |k| about 2^-power: ordinary scores."""
    rng = np.random.default_rng(200 + power)
    c = Cache([50, 17], 1, 16, rng, k=rng.standard_normal((67, 1, 128)) * 2.0 ** -power)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((2, g, 128)) * 2.0 ** power).cuda().to(torch.bfloat16)
    ws = ws_for(2, g)
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws)
    check_decode(c, q, o, lse, g, 0.1, "bf16")
    # the weights of the same step: 1 in all per query head
    w = torch.zeros(2, 1, 64, device="cuda")
    pkc.accumulate_weights(q, lse, d[0], bt, dl, 0.1, w, ws, k_scales=d[1])
    want_w_of_decode(c, q, lse, w, g, 0.1)


def test_decode_of_equal_tiny_queries_and_huge_keys():
    """|q| = 2^-108, |k| = 2^108 throughout: q.k is 128 or -128."""
    rng = np.random.default_rng(1)
    n = 40
    k = np.where(rng.random((n, 1, 1)) < 0.5, -1.0, 1.0) * np.full((n, 1, 128), 2.0 ** 108)
    c = Cache([n], 1, 16, rng, k=k)
    d, bt, dl = c.device()
    q = torch.full((1, 4, 128), 2.0 ** -108, device="cuda", dtype=torch.bfloat16)
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.02, ws_for(1, 4))
    check_decode(c, q, o, lse, 4, 0.02, "bf16")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hkv,batch", [(1, 1), (4, 1300)])
def test_decode_where_every_score_is_near_the_lowest_number(dtype, hkv, batch):
    """All scores -3.3e38 in base 2: equal, finite, so the result is the mean of the values."""
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(1, 70, batch)]
    c = Cache(lens, hkv, 16, rng, k=np.full((sum(lens), hkv, 128), -6 * 2.0 ** 118))
    d, bt, dl = c.device()
    q = torch.ones(batch, 2 * hkv, 128, device="cuda", dtype=DT[dtype])
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.9, ws_for(batch, 2 * hkv))
    o, lse = f64(o), f64(lse)
    np.testing.assert_allclose(lse, -0.9 * 128 * 6 * 2.0 ** 118, rtol=2.0 ** -20)
    eps = torch.finfo(DT[dtype]).eps
    for b in range(batch):
        for h in range(2 * hkv):
            want = c.v[b][:, h // 2].mean(0)
            # sums of up to 70 float32 values, one rounding to the type
            vmax = np.abs(c.v[b][:, h // 2]).max()
            assert np.all(np.abs(o[b, h] - want) <= 2.0 ** -17 * vmax + np.abs(want) * eps / 2 + 2.0 ** -25)


@pytest.mark.parametrize("g", [4, 8])
def test_decode_of_scores_that_are_large_and_finite(g):
    """|q| about 1, |k| = 2^108: q.k of 4e34 is a float32 number; one token has
    the largest score by far and is the result."""
    rng = np.random.default_rng(2)
    n, top = 37, 21
    k = np.full((n, 1, 128), 2.0 ** 108)
    k[:, :, ::2] *= -1
    k[top, 0] = 2.0 ** 110
    c = Cache([n], 1, 16, rng, k=k)
    d, bt, dl = c.device()
    q = torch.ones(1, g, 128, device="cuda", dtype=torch.bfloat16)
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 1.0, ws_for(1, g))
    # the top token's weight is 1 and the others' 0: its values, rounded once
    want = torch.from_numpy(c.v[0][top]).to(torch.bfloat16)
    assert torch.equal(o[0].cpu(), want.expand(g, 128))
    # a float32 sum of 128 products, one rounding to base 2 and one back
    np.testing.assert_allclose(f64(lse), 128 * 2.0 ** 110, rtol=140 * 2.0 ** -24)


def test_heads_of_one_group_with_queries_of_very_different_sizes():
    rng = np.random.default_rng(3)
    g = 4
    c = Cache([100], 1, 16, rng, k=rng.standard_normal((100, 1, 128)) * 2.0 ** -40)
    d, bt, dl = c.device()
    size = np.array([2.0 ** 40, 2.0 ** -120, 2.0 ** 44, 2.0 ** 0])[None, :, None]
    q = torch.from_numpy(rng.standard_normal((1, g, 128)) * size).cuda().to(torch.bfloat16)
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.05, ws_for(1, g))
    check_decode(c, q, o, lse, g, 0.05, "bf16")


# ---------------------------------------------------------------------------
# Scores past 2^24, where a float32 no longer holds every whole number
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("g", [1, 8])
@pytest.mark.parametrize("exp", [10, 18, 19, 20, 21, 22, 24])
def test_decode_of_scores_beyond_whole_float32_numbers(exp, g, sign):
    """Base-2 scores of +- 96 2^exp plus 0, 2, 4, 8, 16 or 32, as far as the type
    tells them apart: every score, difference and probability is exact.

    sm_scale is the float32 ln 2, whose product with the float32 log2 e is 1, so
    q.k is the score in base 2.  Blocks 0 .. 2 make the large part (q 2^(exp / 2),
    k the rest), block 3 one element the small one.
    """
    rng = np.random.default_rng(exp)
    sm = np.float32(np.log(2.0))
    assert sm * np.float32(1.4426950408889634) == 1
    spacing = np.spacing(np.float32(96 * 2.0 ** exp))
    steps = [float(x) for x in (2, 4, 8, 16, 32) if x % spacing == 0] or [0.0]
    lens, offsets = [], []
    for first in (0.0, *steps):  # (of a head's four warps each has 16 tokens of 64)
        for second in (0.0, *steps):
            offsets.append(np.concatenate([np.full(64, first), np.full(64, second), [0.0], rng.choice([0.0, *steps], 70)]))
            lens.append(len(offsets[-1]))
    n = sum(lens)
    small = np.concatenate(offsets)
    k = np.zeros((n, 1, 128))
    k[:, 0, :96] = sign * 2.0 ** (exp - exp // 2)
    k[:, 0, 96] = small
    c = Cache(lens, 1, 16, rng, k=k)
    d, bt, dl = c.device()
    q = torch.zeros(len(lens), g, 128, device="cuda", dtype=torch.float16)
    q[:, :, :96], q[:, :, 96] = 2.0 ** (exp // 2), 1.0
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, float(sm), ws_for(len(lens), g))
    o, lse = f64(o), f64(lse)
    for b, off in enumerate(offsets):
        p = np.exp2(off - off.max())
        want = (p / p.sum()) @ c.v[b][:, 0]
        vmax = np.repeat(np.abs(c.v[b][:, 0]).reshape(-1, 4, 32).max((0, 2)), 32)
        # the exponential and the two-part probabilities (2 2^-20), the sums (2^-18), one rounding to fp16
        tol = (2.0 ** -19 + 2.0 ** -18) * vmax + np.abs(want) * 2.0 ** -11 + 2.0 ** -25
        for h in range(g):
            assert np.all(np.abs(o[b, h] - want) <= tol), (b, h, o[b, h], want)
        want_l = (sign * 96 * 2.0 ** exp + off.max() + np.log2(p.sum())) * np.log(2.0)
        # the score and the logarithm are added, then taken to base e: three roundings, and ln 2's own
        assert np.all(np.abs(lse[b] - want_l) <= abs(want_l) * 2.0 ** -22 + 2.0 ** -18), (b, lse[b], want_l)


# ---------------------------------------------------------------------------
# Values near the smallest and the largest numbers
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("batch,hkv", [(2, 1), (2, 4), (700, 4), (1300, 4)])
@pytest.mark.parametrize("g", [2, 8])
def test_values_near_the_smallest_numbers_keep_their_bits(batch, hkv, g):
    """bf16 values of about 2^-120, in every split of the warps (four, two and
    one per head: the large batch), compared times 2^120."""
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(1, 60, batch)]
    v = (np.abs(rng.standard_normal((sum(lens), hkv, 128))) + 0.5) * 2.0 ** -120
    c = Cache(lens, hkv, 16, rng, v=v)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((batch, hkv * g, 128))).cuda().bfloat16()
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws_for(batch, hkv * g))
    c.v = [x * 2.0 ** 120 for x in c.v]
    check_decode(c, q, o.double() * 2.0 ** 120, lse, g, 0.1, "bf16")


@pytest.mark.parametrize("ps", [16, 5])
def test_values_of_scale_byte_0(ps):
    """Values of 2^-127 and its small multiples, compared times 2^120."""
    rng = np.random.default_rng(7)
    c = Cache([70], 2, ps, rng)
    smallest(c, 2, rng)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((1, 4, 128))).cuda().bfloat16()
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws_for(1, 4))
    ro, rl, sm, vm = ref.attention(f64(q)[0], c.k[0], c.v[0] * 2.0 ** 120, 2, 0.1)
    ot, lt = ref.bounds(ro, rl, sm, vm, 2.0 ** -7)
    # (bf16 results below 2^-126 are multiples of 2^-133: off by 2^-134 at most)
    assert np.all(np.abs(f64(o)[0] * 2.0 ** 120 - ro) <= ot + 2.0 ** -14)
    assert np.all(np.abs(f64(lse)[0] - rl) <= lt)


@pytest.mark.parametrize("size", [2.0 ** -100, 1e37])
def test_values_of_one_sign_in_split_requests(size):
    """Values of about `size`, all positive: their mean over a request that a
    plan splits into many chunks is of that size too."""
    rng = np.random.default_rng(5)
    lens, hkv, g, ctas = [6000, 40, 0], 1, 4, 148
    c = Cache(lens, hkv, 16, rng, v=(np.abs(rng.standard_normal((6040, hkv, 128))) + 0.5) * size)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((3, hkv * g, 128))).cuda().bfloat16()
    ws, plan = ws_for(3, hkv * g, ctas), pkc.plan(lens, ctas)
    pkc.plan_upload(plan, ws)
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws, plan_buf=plan)
    c.v = [x / size for x in c.v]
    check_decode(c, q, o.double() / size, lse, g, 0.1, "bf16")
