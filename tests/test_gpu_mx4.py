"""The mx4 paged cache on the GPU: quantising append, read-back and decode
against the float64 reference of the format (mx4_reference)."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
import paged_kv_cascade_gb300 as pkc

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7}


def ws_for(B, Hq, ctas=0):
    ws = torch.empty(pkc.workspace_size(B, Hq, ctas, 0), dtype=torch.uint8, device="cuda")
    pkc.workspace_init(ws)
    return ws


def f64(t):
    return t.detach().cpu().double().numpy()


def table_for(lens, ps, rng, spare=2):
    """Block table (-1 unused) over a permuted pool with `spare` pages of nobody."""
    need = [(n + ps - 1) // ps for n in lens]
    P = sum(need) + spare
    perm = rng.permutation(P).astype(np.int32)
    bt = np.full((len(lens), max(1, max(need, default=1))), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        bt[b, :k] = perm[at:at + k]
        at += k
    return bt, P


def indptr_of(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Cache:
    """An mx4 cache of random bytes (slots of nobody hold NaN scales) filled
    with quantised values for each request."""

    def __init__(self, lens, hkv, ps, rng, k=None, v=None, spare=2):
        self.lens, self.hkv, self.ps = list(lens), hkv, ps
        self.bt, self.P = table_for(lens, ps, rng, spare)
        shape = (self.P, ps, hkv)
        self.pools = [rng.integers(0, 256, shape + (64,)).astype(np.uint8), np.full(shape + (4,), 255, np.uint8),
                      rng.integers(0, 256, shape + (64,)).astype(np.uint8), np.full(shape + (4,), 255, np.uint8)]
        n = sum(lens)
        k = rng.standard_normal((n, hkv, 128)) if k is None else k
        v = rng.standard_normal((n, hkv, 128)) if v is None else v
        at = 0
        self.k, self.v = [], []
        for b, m in enumerate(lens):
            for j, x in ((0, k), (2, v)):
                c, s = ref.quantise(x[at:at + m])
                for t in range(m):
                    page, slot = self.bt[b, t // ps], t % ps
                    self.pools[j][page, slot], self.pools[j + 1][page, slot] = c[t], s[t]
                (self.k if j == 0 else self.v).append(ref.values(c, s))
            at += m

    def device(self):
        self.d = [cuda(p) for p in self.pools]
        return self.d, cuda(self.bt), cuda(np.asarray(self.lens, np.int32))


def check_decode(cache, q, o, lse, g, scale, dtype):
    o, lse, qd = f64(o), f64(lse), f64(q)
    for b in range(len(cache.lens)):
        ro, rl, sm, vm = ref.attention(qd[b], cache.k[b], cache.v[b], g, scale)
        ot, lt = ref.bounds(ro, rl, sm, vm, EPS[dtype])
        if cache.lens[b] == 0:
            assert np.all(o[b] == 0) and np.all(np.isneginf(lse[b]))
            continue
        assert np.all(np.abs(o[b] - ro) <= ot), (b, np.max(np.abs(o[b] - ro) / ot))
        assert np.all(np.abs(lse[b] - rl) <= lt), (b, np.max(np.abs(lse[b] - rl) / lt))


# ---------------------------------------------------------------------------
# Append and read-back
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_16_bit_pattern_quantises_as_defined(dtype):
    rng = np.random.default_rng(1)
    bits = rng.permutation(65536).astype(np.uint16)
    finite = (bits & (0x7c00 if dtype == "f16" else 0x7f80)) != (0x7c00 if dtype == "f16" else 0x7f80)
    # blocks of neighbouring magnitudes, so that all of a block's codes occur, and blocks of anything
    near = np.sort(bits[finite] & 0x7fff)
    near = near[: len(near) // 128 * 128] | (rng.integers(0, 2, len(near) // 128 * 128).astype(np.uint16) << 15)
    rows = np.concatenate([near, bits]).astype(np.uint16).reshape(-1, 1, 128)
    T = rows.shape[0]
    x = torch.from_numpy(rows.view(np.int16)).cuda().view(DT[dtype])
    ps = 16
    P = (T + ps - 1) // ps
    pools = [torch.zeros((P, ps, 1, n), dtype=torch.uint8, device="cuda") for n in (64, 4, 64, 4)]
    bt = torch.arange(P, dtype=torch.int32, device="cuda")[None]
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = ws_for(1, 1)
    ip = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    pkc.append_kv_mx4(x, x.flip(0).contiguous(), ip, *pools, bt, lens, ws)
    k, v = pkc.gather_kv_mx4(*pools, bt, torch.zeros_like(lens), ip, T, ws, dtype=DT[dtype])
    assert pkc.device_status(ws) == pkc.PKC_OK and lens.item() == T
    with np.errstate(invalid="ignore"):
        codes, scales = ref.quantise(f64(x))
    got_c, got_s = pools[0].cpu().numpy().reshape(-1, 1, 64)[:T], pools[1].cpu().numpy().reshape(-1, 1, 4)[:T]
    np.testing.assert_array_equal(got_s, scales)
    np.testing.assert_array_equal(got_c, codes)
    np.testing.assert_array_equal(pools[2].cpu().numpy().reshape(-1, 1, 64)[:T], codes[::-1])
    # read back: the values rounded to the type (torch's rounding of the exact float32 value)
    want = torch.from_numpy(ref.values(codes, scales)).float().to(DT[dtype])
    assert torch.equal(torch.nan_to_num(k.cpu(), nan=123.0), torch.nan_to_num(want, nan=123.0))
    assert torch.equal(torch.nan_to_num(v.cpu().flip(0), nan=123.0), torch.nan_to_num(want, nan=123.0))


@pytest.mark.parametrize("hkv,ps,old,new", [
    (1, 1, [0, 3, 0], [1, 2, 0]),
    (8, 16, [15, 16, 0, 31, 5, 47], [1, 1, 1, 1, 1, 1]),
    (3, 7, [0, 13, 6, 200], [0, 1, 15, 500]),
    (2, 24, [23, 0], [1000, 1]),
    (4, 64, [0] * 40, [0] * 39 + [3]),
])
def test_append_writes_the_next_slots_and_nothing_else(hkv, ps, old, new):
    rng = np.random.default_rng(hkv * 100 + ps)
    total = sum(new)
    bt, P = table_for([a + b for a, b in zip(old, new)], ps, rng)
    pools = [rng.integers(0, 256, (P, ps, hkv, n)).astype(np.uint8) for n in (64, 4, 64, 4)]
    kn, vn = (torch.from_numpy(rng.standard_normal((total + 3, hkv, 128)) * 3).cuda().to(torch.bfloat16) for _ in "kv")
    d = [cuda(p) for p in pools]
    lens, ip, ws = cuda(np.asarray(old, np.int32)), cuda(indptr_of(new)), ws_for(len(old), hkv)
    for rep in range(2):  # the second call finds the workspace's counter as the first left it
        lens.copy_(cuda(np.asarray(old, np.int32)))
        pkc.append_kv_mx4(kn, vn, ip, *d, cuda(bt), lens, ws)  # three rows behind the last request
    assert pkc.device_status(ws) == pkc.PKC_OK
    np.testing.assert_array_equal(lens.cpu().numpy(), np.add(old, new))
    row = 0
    for b, n in enumerate(new):
        for i in range(n):
            t = old[b] + i
            for j, x in ((0, kn), (2, vn)):
                c, s = ref.quantise(f64(x[row]))
                pools[j][bt[b, t // ps], t % ps] = c
                pools[j + 1][bt[b, t // ps], t % ps] = s
            row += 1
    for got, want in zip(d, pools):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_append_without_a_page_and_with_a_bad_range():
    rng = np.random.default_rng(3)
    old, new = [3, 16, 9, 30], [2, 3, 1, 4]
    bt, P = table_for([a + b for a, b in zip(old, new)], 16, rng)
    bt[1, 1] = -1   # request 1's tokens 16 .. 18
    bt[3, 2] = P    # request 3's tokens 32, 33 (its first two are in page 1)
    d = [torch.zeros((P, 16, 2, n), dtype=torch.uint8, device="cuda") for n in (64, 4, 64, 4)]
    x = torch.randn(sum(new), 2, 128, device="cuda").half()
    lens, ws = cuda(np.asarray(old, np.int32)), ws_for(4, 2)
    pkc.append_kv_mx4(x, x, cuda(indptr_of(new)), *d, cuda(bt), lens, ws)
    assert pkc.device_status(ws) == 4  # PKC_ERR_BLOCK_TABLE
    assert lens.tolist() == [5, 16, 10, 30]
    # ranges that run backwards, past the rows, from below 0: no length changes
    bt, P = table_for([20] * 4, 16, rng)
    d = [torch.zeros((P, 16, 2, n), dtype=torch.uint8, device="cuda") for n in (64, 4, 64, 4)]
    for ranges in ([0, 4, 2, 6, 10], [0, 1, 2, 3, 11], [-3, 1, 2, 3, 4], [0, 2 ** 31 - 1, 5, 6, 7]):
        lens = cuda(np.full(4, 2, np.int32))
        pkc.append_kv_mx4(x, x, cuda(np.array(ranges, np.int32)), *d, cuda(bt), lens, ws)
        assert pkc.device_status(ws) in (4, 7)  # PKC_ERR_PLAN (or first a token past the table)
        assert lens.tolist() == [2, 2, 2, 2]
    # and the workspace's counters are clean again
    lens = cuda(np.full(4, 2, np.int32))
    pkc.append_kv_mx4(x, x, cuda(indptr_of(new)), *d, cuda(bt), lens, ws)
    assert pkc.device_status(ws) == pkc.PKC_OK and lens.tolist() == [4, 5, 3, 6]


def test_gather_leaves_rows_of_nobody_and_zeroes_rows_without_a_page():
    rng = np.random.default_rng(4)
    c = Cache([40, 20, 7], 3, 8, rng)
    d, bt, _ = c.device()
    bt[1, 1] = -1  # request 1's tokens 8 .. 15
    ip = cuda(np.array([2, 12, 22, 22], np.int32))  # rows 0, 1 and 22 .. belong to nobody
    first = cuda(np.array([30, 5, 3], np.int32))
    k = torch.full((25, 3, 128), 9.0, device="cuda", dtype=torch.bfloat16)
    v = torch.full_like(k, 9.0)
    ws = ws_for(3, 3)
    pkc.gather_kv_mx4(*d, bt, first, ip, 25, ws, k=k, v=v)
    assert pkc.device_status(ws) == 4
    for got, val in ((k, c.k), (v, c.v)):
        want = np.full((25, 3, 128), 9.0)
        want[2:12] = val[0][30:40]
        want[12:22] = val[1][5:15]
        want[15:22] = 0.0  # tokens 8 .. 14
        assert torch.equal(got.cpu(), torch.from_numpy(want).float().to(torch.bfloat16))


# ---------------------------------------------------------------------------
# Decode
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hkv,g,ps", [(1, 1, 16), (2, 8, 5), (3, 2, 1), (4, 4, 8), (8, 4, 16), (8, 1, 48)])
def test_decode_without_a_plan(dtype, hkv, g, ps):
    rng = np.random.default_rng(hkv * 10 + g)
    c = Cache([0, 1, 15, 16, 17, 63, 130, 301], hkv, ps, rng)
    d, bt, lens = c.device()
    q = torch.from_numpy(rng.standard_normal((len(c.lens), hkv * g, 128)) * 2).cuda().to(DT[dtype])
    ws = ws_for(len(c.lens), hkv * g)
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, lens, 0.09, ws)
    assert pkc.device_status(ws) == pkc.PKC_OK
    check_decode(c, q, o, lse, g, 0.09, dtype)


@pytest.mark.parametrize("schedule", ["dynamic", "static"])
@pytest.mark.parametrize("dtype,hkv,g,ps,ctas,lens", [
    ("f16", 8, 4, 16, 40, [700, 0, 33, 1, 2048, 15]),
    ("bf16", 4, 8, 16, 148, [3001, 5]),
    ("f16", 1, 2, 6, 7, [100, 1000, 0]),
    ("bf16", 2, 1, 128, 300, [4000]),
    ("f16", 16, 1, 16, 20, [64] * 33),
])
def test_planned_decode(schedule, dtype, hkv, g, ps, ctas, lens):
    rng = np.random.default_rng(ctas)
    c = Cache(lens, hkv, ps, rng)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((len(lens), hkv * g, 128)) * 2).cuda().to(DT[dtype])
    ws = ws_for(len(lens), hkv * g, ctas)
    plan = pkc.plan(lens, ctas)
    pkc.plan_upload(plan, ws)
    try:
        pkc.set_decode_schedule(schedule)
        outs = [pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws, plan_buf=plan) for _ in range(3)]
    finally:
        pkc.set_decode_schedule("dynamic")
    assert pkc.device_status(ws) == pkc.PKC_OK
    check_decode(c, q, *outs[0], g, 0.1, dtype)
    for o, lse in outs[1:]:  # the same bits every time
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("spread", [3, 12, 40])
def test_decode_with_scales_far_apart(spread):
    """Block scales of K and V that differ by up to 2^spread between tokens,
    queries whose elements do too."""
    rng = np.random.default_rng(spread)
    lens, hkv, g = [260, 37], 2, 4
    n = sum(lens)
    e = lambda: np.exp2(rng.integers(-spread, 1, (n, hkv, 4)))  # noqa: E731
    k = rng.standard_normal((n, hkv, 128)) * np.repeat(e(), 32, -1)
    v = rng.standard_normal((n, hkv, 128)) * np.repeat(e(), 32, -1)
    c = Cache(lens, hkv, 16, rng, k=k, v=v)
    d, bt, dl = c.device()
    q = rng.standard_normal((2, hkv * g, 128)) * np.exp2(rng.integers(-min(spread, 14), 1, (2, hkv * g, 128)))
    for dtype in ("f16", "bf16"):
        qd = torch.from_numpy(q).cuda().to(DT[dtype])
        ws = ws_for(2, hkv * g)
        o, lse = pkc.paged_decode_state_mx4(qd, *d, bt, dl, 0.3, ws)
        check_decode(c, qd, o, lse, g, 0.3, dtype)


@pytest.mark.parametrize("mag", [2.0 ** -100, 2.0 ** 100])
def test_decode_of_very_small_and_very_large_bf16_queries(mag):
    """bf16 queries far outside fp16's range, keys that bring the scores back."""
    rng = np.random.default_rng(7)
    lens, hkv, g = [50], 1, 2
    c = Cache(lens, hkv, 16, rng, k=rng.standard_normal((50, 1, 128)) / mag)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((1, 2, 128)) * mag).cuda().to(torch.bfloat16)
    ws = ws_for(1, 2)
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws)
    check_decode(c, q, o, lse, g, 0.1, "bf16")


@pytest.mark.parametrize("hkv", [1, 4])
def test_decode_of_values_near_the_largest_float(hkv):
    """bf16 values of 1e37: their weighted sum stays finite, as it is a mean."""
    rng = np.random.default_rng(10)
    lens, g = [300, 33], 4
    c = Cache(lens, hkv, 16, rng, v=rng.standard_normal((333, hkv, 128)) * 1e37)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((2, hkv * g, 128))).cuda().bfloat16()
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws_for(2, hkv * g))
    check_decode(c, q, o, lse, g, 0.1, "bf16")


@pytest.mark.parametrize("hkv", [1, 4])
def test_decode_of_tiny_values(hkv):
    """bf16 values of 2^-100 keep their bits (compared times 2^100)."""
    rng = np.random.default_rng(13)
    lens, g = [300, 33], 2
    c = Cache(lens, hkv, 16, rng, v=rng.standard_normal((333, hkv, 128)) * 2.0 ** -100)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((2, hkv * g, 128))).cuda().bfloat16()
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws_for(2, hkv * g))
    c.v = [v * 2.0 ** 100 for v in c.v]
    check_decode(c, q, o.double() * 2.0 ** 100, lse, g, 0.1, "bf16")


def test_decode_of_large_scores_moves_the_reference():
    """Scores that rise along the cache by hundreds: earlier tokens' weights vanish."""
    rng = np.random.default_rng(8)
    n = 200
    k = rng.standard_normal((n, 1, 128)) * np.linspace(0.1, 40, n)[:, None, None]
    c = Cache([n], 1, 16, rng, k=k)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((1, 8, 128)) * 3).cuda().half()
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 1.0, ws_for(1, 8))
    check_decode(c, q, o, lse, 8, 1.0, "f16")


def test_nan_blocks_reach_the_output_of_their_request_only():
    rng = np.random.default_rng(9)
    lens = [40, 40, 40]
    n = sum(lens)
    k, v = rng.standard_normal((n, 2, 128)), rng.standard_normal((n, 2, 128))
    k[10, 0, 5] = np.nan           # request 0, head 0: every output of that head
    v[50, 1, 70] = np.inf          # request 1, head 1: dims 64 .. 95
    c = Cache(lens, 2, 16, rng, k=k, v=v)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((3, 4, 128))).cuda().half()
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws_for(3, 4))
    o, lse = f64(o), f64(lse)
    want_o, want_l = np.zeros((3, 4, 128), bool), np.zeros((3, 4), bool)
    want_o[0, :2], want_l[0, :2] = True, True
    want_o[1, 2:, 64:96] = True
    np.testing.assert_array_equal(np.isnan(o), want_o)
    np.testing.assert_array_equal(np.isnan(lse), want_l)


def test_decode_reports_bad_pages_and_leaves_their_tokens_out():
    rng = np.random.default_rng(10)
    c = Cache([50, 40], 2, 16, rng)
    d, bt, dl = c.device()
    bt[0, 1], bt[1, 0] = c.P, -5
    q = torch.from_numpy(rng.standard_normal((2, 4, 128))).cuda().half()
    ws = ws_for(2, 4)
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws)
    assert pkc.device_status(ws) == 4
    drop = [np.r_[0:16, 32:50], np.r_[16:40]]
    for x in (c.k, c.v):
        for b in range(2):
            x[b] = x[b][drop[b]]
    check_decode(c, q, o, lse, 2, 0.1, "f16")
    # more tokens than the table holds: reported, the table's tokens are used
    c = Cache([32], 1, 16, rng)
    d, bt, dl = c.device()
    ws = ws_for(1, 1)
    q = q[:1, :1].contiguous()
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl + 1000, 0.1, ws)
    assert pkc.device_status(ws) == 4
    check_decode(c, q, o, lse, 1, 0.1, "f16")


def test_plan_that_was_not_uploaded_is_reported():
    rng = np.random.default_rng(11)
    c = Cache([50, 40], 2, 16, rng)
    d, bt, dl = c.device()
    ws = ws_for(2, 4, 8)
    ws[256:4096] = 0
    pkc.paged_decode_state_mx4(torch.zeros(2, 4, 128, device="cuda").half(), *d, bt, dl, 0.1, ws,
                               plan_buf=pkc.plan([50, 40], 8))
    assert pkc.device_status(ws) == 7


def test_host_plan_that_is_not_the_uploaded_one():
    """The join follows the uploaded plan: a host plan of the same sizes with
    other splits changes no result."""
    rng = np.random.default_rng(21)
    lens, hkv, g, ctas = [900, 10, 0, 400], 2, 4, 16
    c = Cache(lens, hkv, 16, rng)
    d, bt, dl = c.device()
    q = torch.from_numpy(rng.standard_normal((4, hkv * g, 128))).cuda().half()
    ws = ws_for(4, hkv * g, ctas)
    plan, other = pkc.plan(lens, ctas), pkc.plan([5, 5, 5, 5], ctas)
    assert plan.size == other.size
    pkc.plan_upload(plan, ws)
    o, lse = pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws, plan_buf=other)
    assert pkc.device_status(ws) == pkc.PKC_OK
    check_decode(c, q, o, lse, g, 0.1, "f16")
    # and an uploaded plan of other lengths is reported
    pkc.plan_upload(other, ws)
    pkc.paged_decode_state_mx4(q, *d, bt, dl, 0.1, ws, plan_buf=plan)
    assert pkc.device_status(ws) == 7


def test_append_then_decode_in_a_captured_graph_on_another_stream():
    """Prompt, then steps of one token: each replay appends the tokens in the
    static buffers and decodes; results as without the graph."""
    rng = np.random.default_rng(12)
    lens, hkv, g, ps, steps = [5, 0, 31, 16], 4, 4, 16, 3
    B = len(lens)
    bt, P = table_for([n + steps for n in lens], ps, rng)
    xs = [torch.from_numpy(rng.standard_normal((sum(lens) if i == 0 else B, hkv, 128))).cuda().half()
          for i in range(2 * (steps + 1))]
    xs = [xs[0], xs[0] * 0.5] + xs[2:]
    xs = [x if i < 2 or x.shape[0] == B else x[:B].contiguous() for i, x in enumerate(xs)]
    qs = torch.from_numpy(rng.standard_normal((steps, B, hkv * g, 128))).cuda().half()
    table, one = cuda(bt), torch.arange(B + 1, dtype=torch.int32, device="cuda")

    def fresh():
        d = [torch.zeros((P, ps, hkv, n), dtype=torch.uint8, device="cuda") for n in (64, 4, 64, 4)]
        dl, ws = torch.zeros(B, dtype=torch.int32, device="cuda"), ws_for(B, hkv * g)
        pkc.append_kv_mx4(xs[0], xs[1], cuda(indptr_of(lens)), *d, table, dl, ws)
        return d, dl, ws

    d, dl, ws = fresh()
    want = []
    for i in range(steps):
        pkc.append_kv_mx4(xs[2 + 2 * i], xs[3 + 2 * i], one, *d, table, dl, ws)
        want.append(pkc.paged_decode_state_mx4(qs[i], *d, table, dl, 0.1, ws))
    d2, dl2, ws2 = fresh()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k, v, q = xs[2].clone(), xs[3].clone(), qs[0].clone()
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pkc.append_kv_mx4(k, v, one, *d2, table, dl2, ws2)
        pkc.paged_decode_state_mx4(q, *d2, table, dl2, 0.1, ws2, o=o, lse=lse)
    for i in range(steps):
        k.copy_(xs[2 + 2 * i]), v.copy_(xs[3 + 2 * i]), q.copy_(qs[i])
        graph.replay()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    assert dl2.tolist() == [n + steps for n in lens]
    assert pkc.device_status(ws2) == pkc.PKC_OK
    for a, b in zip(d, d2):
        assert torch.equal(a, b)


def test_slots_past_two_gigabytes():
    """Pools of more than 2^31 bytes: the last pages."""
    rng = np.random.default_rng(13)
    ps, hkv, lens = 16, 8, [30]
    P = (1 << 31) // (ps * hkv * 64) + 40
    pools = [torch.zeros((P, ps, hkv, n), dtype=torch.uint8, device="cuda") for n in (64, 4, 64, 4)]
    bt = torch.tensor([[P - 1, P - 3]], dtype=torch.int32, device="cuda")
    x = torch.from_numpy(rng.standard_normal((2, 30, hkv, 128))).cuda().half()
    dl, ws = torch.zeros(1, dtype=torch.int32, device="cuda"), ws_for(1, hkv)
    ip = torch.tensor([0, 30], dtype=torch.int32, device="cuda")
    pkc.append_kv_mx4(x[0], x[1], ip, *pools, bt, dl, ws)
    c = Cache(lens, hkv, ps, rng, k=f64(x[0]), v=f64(x[1]))
    k, v = pkc.gather_kv_mx4(*pools, bt, torch.zeros_like(dl), ip, 30, ws)
    np.testing.assert_array_equal(f64(k), c.k[0])
    np.testing.assert_array_equal(f64(v), c.v[0])
    q = torch.from_numpy(rng.standard_normal((1, hkv, 128))).cuda().half()
    o, lse = pkc.paged_decode_state_mx4(q, *pools, bt, dl, 0.1, ws)
    check_decode(c, q, o, lse, 1, 0.1, "f16")
    assert pkc.device_status(ws) == pkc.PKC_OK


def test_binding_refuses_wrong_device_tensors():
    """Every tensor of every call: another dtype, another shape, strides."""
    u8, i32, f32 = torch.uint8, torch.int32, torch.float32
    z = lambda *s, d=u8: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    pools = [z(4, 16, 2, 64), z(4, 16, 2, 4), z(4, 16, 2, 64), z(4, 16, 2, 4)]
    bt, lens, ws, ip = z(3, 4, d=i32), z(3, d=i32), ws_for(3, 4), z(4, d=i32)
    x, q, lse, w = z(5, 2, 128, d=torch.float16), z(3, 4, 128, d=torch.float16), z(3, 4, d=f32), z(3, 2, 64, d=f32)
    k16, keep = z(4, 16, 2, 128, d=torch.float16), z(3, 2, 8, d=i32)
    calls = [
        (pkc.append_kv_mx4, [x, x, ip, *pools, bt, lens, ws]),
        (pkc.gather_kv_mx4, [*pools, bt, lens, ip, 5, ws]),
        (pkc.paged_decode_state_mx4, [q, *pools, bt, lens, 0.1, ws]),
        (pkc.accumulate_weights, [q, lse, k16, bt, lens, 0.1, w, ws]),
        (pkc.evict_select, [w, lens, 8, 1, 1, ws]),
        (pkc.evict_compact, [keep, k16, k16.clone(), bt, lens, ws]),
    ]
    for fn, args in calls:
        fn(*args)  # (lengths 0: nothing happens)
        for i, t in enumerate(args):
            if not isinstance(t, torch.Tensor):
                continue
            doubled = torch.zeros(t.shape[:-1] + (2 * t.shape[-1],), dtype=t.dtype, device="cuda")[..., ::2]
            bad = [t.to(torch.float64), t[None], t.cpu(), doubled, "tensor", None]
            # one more row: refused but where that tensor alone gives the size (new rows, a pool's pages)
            alone = (fn is pkc.append_kv_mx4 and i == 0) or (fn is pkc.accumulate_weights and i == 2)
            if t is not ws and not alone:
                bad.append(torch.cat([t, t[:1]]))
            for b in bad:
                with pytest.raises((TypeError, ValueError, AttributeError)):
                    fn(*args[:i], b, *args[i + 1:])
                    print(fn.__name__, i, b)  # (shown when nothing was raised)
    assert pkc.device_status(ws) == pkc.PKC_OK
    with pytest.raises((TypeError, ValueError)):
        pkc.gather_kv_mx4(*pools, bt, lens, ip, 5, ws, dtype=f32)
    with pytest.raises(ValueError):
        pkc.gather_kv_mx4(*pools, bt, lens, ip, -1, ws)
    with pytest.raises(ValueError):
        pkc.evict_select(w, lens, 8, 5, 4, ws)
    with pytest.raises(ValueError):
        pkc.evict_compact(keep, pools[0], pools[2], bt, lens, ws, k_scales=pools[1])
    for bad in (dict(decay=1.5), dict(decay=float("nan")), dict(k_scale=2.0)):
        with pytest.raises(pkc.PkcError):
            pkc.accumulate_weights(q, lse, k16, bt, lens, 0.1, w, ws, **bad)
