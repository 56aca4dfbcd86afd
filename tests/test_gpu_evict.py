"""Eviction on the GPU: accumulated attention weights against float64, the
selection and the move against plain numpy, and the three together with
decode and append over every kind of cache."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
import paged_kv_cascade_gb300 as pkc
from test_gpu_mx4 import DT, cuda, f64, table_for, ws_for

pytestmark = pytest.mark.gpu

KINDS = ["f16", "bf16", "e4m3", "mx4", "mx4_bf16q"]
E4M3 = torch.float8_e4m3fn


def q_type(kind):
    return torch.bfloat16 if kind in ("bf16", "mx4_bf16q") else torch.float16


class Paged:
    """Paged K and V of one kind on the device and their float64 values per request."""

    def __init__(self, kind, lens, hkv, ps, rng, room=0, k=None):
        self.kind, self.lens, self.hkv, self.ps = kind, list(lens), hkv, ps
        self.mx4 = kind.startswith("mx4")
        self.bt_host, self.P = table_for([n + room for n in lens], ps, rng)
        shape = (self.P, ps, hkv, 128)
        self.k_scale = 0.5 if kind == "e4m3" else 1.0
        t, self.scales = [], [None, None]
        for i in range(2):
            x = torch.from_numpy(rng.standard_normal(shape) if k is None or i else np.resize(k, shape))
            if self.mx4:
                c, s = ref.quantise(x.numpy())
                t.append(cuda(c))
                self.scales[i] = cuda(s)
            elif kind == "e4m3":
                t.append(x.float().to(E4M3).view(torch.uint8).cuda())
            else:
                t.append(x.to(DT[kind]).cuda())
        self.k, self.v = t
        self.bt, self.dl = cuda(self.bt_host), cuda(np.asarray(lens, np.int32))

    def pool(self, i):
        """float64 pool [P, ps, Hkv, 128] of K (0) or V (1)."""
        x = (self.k, self.v)[i]
        if self.mx4:
            return ref.values(x.cpu().numpy(), self.scales[i].cpu().numpy())
        if self.kind == "e4m3":
            return x.view(E4M3).float().cpu().double().numpy() * (self.k_scale if i == 0 else 1.0)
        return f64(x)

    def rows(self, i, b, n):
        return ref.request_rows(self.pool(i), self.bt_host[b], n, self.ps)

    def accumulate(self, q, lse, scale, w, ws, **kw):
        return pkc.accumulate_weights(q, lse, self.k, self.bt, self.dl, scale, w, ws, k_scale=self.k_scale,
                                      k_scales=self.scales[0], **kw)

    def compact(self, keep, ws, w=None):
        pkc.evict_compact(keep, self.k, self.v, self.bt, self.dl, ws, weights=w, k_scales=self.scales[0],
                          v_scales=self.scales[1])

    def decode(self, q, scale, ws):
        if self.mx4:
            return pkc.paged_decode_state_mx4(q, self.k, self.scales[0], self.v, self.scales[1], self.bt, self.dl, scale, ws)
        if self.kind == "e4m3":
            return pkc.paged_decode_state_fp8(q, self.k, self.v, self.bt, self.dl, scale, ws, k_scale=self.k_scale)
        return pkc.paged_decode_state(q, self.k, self.v, self.bt, self.dl, scale, ws)


def want_weights(c, q, lse, scale, w, decay, g):
    """float64 weights and their error bounds.

    The exponent sm q.k - lse carries a float32 sum of 128 products (137
    half-steps of scale * sum |q k|) and two roundings of |lse| in base 2; the
    exponential adds 2^-21, the sums and the decay product 2^-22 of the result.
    """
    qd, ld = f64(q), f64(lse)
    want, tol = w.copy(), np.zeros_like(w)
    for b, n in enumerate(c.lens):
        k = c.rows(0, b, n)
        for h in range(c.hkv):
            new, err = np.zeros(n), np.zeros(n)
            for i in range(h * g, h * g + g):
                if np.isneginf(ld[b, i]):
                    continue
                s = scale * (k[:, h] @ qd[b, i])
                mag = scale * (np.abs(k[:, h]) @ np.abs(qd[b, i]))
                p = np.exp(s - ld[b, i])
                new += p
                err += p * (137 * 2.0 ** -24 * mag + abs(ld[b, i]) * 2.0 ** -22 + 2.0 ** -21)
            want[b, h, :n] = (decay * w[b, h, :n] if decay else 0.0) + new
            tol[b, h, :n] = 1.01 * err + 2.0 ** -22 * np.abs(want[b, h, :n]) + 2.0 ** -126
    return want, tol


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hkv,g,ps,lens", [
    (1, 1, 16, [0, 1, 15, 16, 17, 33]),
    (2, 8, 5, [300, 7]),
    (3, 2, 1, [65, 0, 1]),
    (8, 4, 16, [1000, 129, 1]),
    (4, 1, 64, [2500]),
])
def test_accumulated_weights(kind, hkv, g, ps, lens):
    rng = np.random.default_rng(len(lens) * 10 + g)
    c = Paged(kind, lens, hkv, ps, rng)
    B, W = len(lens), c.bt_host.shape[1] * ps + 3
    q = torch.from_numpy(rng.standard_normal((B, hkv * g, 128)) * 2).cuda().to(q_type(kind))
    lse = torch.from_numpy(np.stack([ref.attention(f64(q)[b], c.rows(0, b, n), c.rows(1, b, n), g, 0.09)[1]
                                     for b, n in enumerate(lens)])).float().cuda()
    ws = ws_for(B, hkv * g)
    w0 = rng.random((B, hkv, W)).astype(np.float32)
    for decay in (1.0, 0.5, 0.0):
        w = cuda(w0)
        if decay == 0.0:  # the old weights are not read
            w[:, :, : max(lens)] = torch.nan
            for b, n in enumerate(lens):
                w[b, :, n:] = cuda(w0[b, :, n:])
        c.accumulate(q, lse, 0.09, w, ws, decay=decay)
        want, tol = want_weights(c, q, lse, 0.09, w0.astype(np.float64), decay, g)
        got = f64(w)
        assert np.all(np.abs(got - want) <= tol), np.nanmax(np.abs(got - want) - tol)
        for b, n in enumerate(lens):  # nothing behind the length
            np.testing.assert_array_equal(got[b, :, n:], w0[b, :, n:])
    # one decay-0 step: a head's weights sum to its g heads' 1 each
    for b, n in enumerate(lens):
        if n:
            np.testing.assert_allclose(got[b, :, :n].sum(-1), g, rtol=1e-4)
    assert pkc.device_status(ws) == pkc.PKC_OK


def test_weights_with_empty_heads_infinite_keys_and_missing_pages():
    rng = np.random.default_rng(5)
    k = np.full((1, 1, 1, 128), 0.25)
    c = Paged("f16", [40, 24], 1, 8, rng, k=k)
    q = torch.full((2, 2, 128), -1.0, device="cuda").half()
    c.k[c.bt_host[0, 0], 3, 0, 7] = float("inf")   # q.k = -inf: weight 0, and no other column's NaN
    lse = torch.tensor([[np.log(2.0), -np.inf], [-np.inf, -np.inf]], device="cuda").float()
    c.bt[0, 2] = -1
    ws, w = ws_for(2, 2), torch.full((2, 1, 64), 7.0, device="cuda")
    c.accumulate(q, lse, 0.01, w, ws, decay=0.5)
    assert pkc.device_status(ws) == 4
    got = w.cpu().numpy()
    p = np.exp(0.01 * -32.0) / 2
    want = np.full(64, 7.0)
    want[:40] = 3.5 + p
    want[3], want[16:24] = 3.5, 7.0
    np.testing.assert_allclose(got[0, 0], want, rtol=2.0 ** -20)
    np.testing.assert_allclose(got[1, 0], [3.5] * 24 + [7.0] * 40)
    # a weights row shorter than the request, a table shorter than it
    w = torch.full((2, 1, 10), 1.0, device="cuda")
    c.accumulate(q, lse, 0.01, w, ws, decay=0.5)
    assert pkc.device_status(ws) in (4, 7)
    assert np.all(w.cpu().numpy()[1] == 0.5)


# ---------------------------------------------------------------------------
# Select
# ---------------------------------------------------------------------------

def select_plain(w, n, budget, sinks, recent):
    """One row: sort by (weight descending, slot ascending)."""
    if n <= budget:
        return np.concatenate([np.arange(n), np.full(budget - n, -1)]).astype(np.int32)
    mid = np.arange(sinks, n - recent)
    x = w[mid].astype(np.float64)
    x = np.where(np.isnan(x), np.inf, x)
    nan_first = np.where(np.isnan(w[mid]), 0, 1)
    order = np.lexsort((mid, -x, nan_first))
    top = np.sort(mid[order[: budget - sinks - recent]])
    return np.concatenate([np.arange(sinks), top, np.arange(n - recent, n)]).astype(np.int32)


def rows_of(kind, shape, rng):
    if kind == "spread":
        return np.exp(3 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "equal":
        return np.full(shape, 0.25, np.float32)
    if kind == "few values":
        return rng.integers(0, 4, shape).astype(np.float32) / 8
    if kind == "mostly zero":
        return np.where(rng.random(shape) < 0.95, 0.0, rng.random(shape)).astype(np.float32)
    if kind == "last bits":
        return (np.float32(1.0).view(np.uint32) + rng.integers(0, 700, shape).astype(np.uint32)).view(np.float32)
    x = rng.standard_normal(shape).astype(np.float32)
    flat = x.reshape(-1)
    odd = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3.4e38, -3.4e38], np.float32)
    pick = rng.random(flat.size) < 0.4
    flat[pick] = odd[rng.integers(0, len(odd), pick.sum())]
    return x


@pytest.mark.parametrize("kind", ["spread", "equal", "few values", "mostly zero", "last bits", "odd values"])
@pytest.mark.parametrize("hkv,lens,budget,sinks,recent", [
    (1, [0, 1, 5, 6, 7, 50], 6, 1, 2),
    (3, [1000, 31, 999], 100, 0, 1),
    (2, [4000, 700, 513], 512, 4, 508),
    (2, [4000, 700, 513], 512, 0, 0),
    (2, [70000, 200], 1024, 4, 64),
    (1, [100001], 33333, 3, 10000),
    (1, [9], 1, 0, 1),
    (1, [9], 1, 0, 0),
    (80, [5000, 4097], 1000, 4, 100),
    (80, [30000, 26000], 5000, 4, 100),
])
def test_select(kind, hkv, lens, budget, sinks, recent):
    rng = np.random.default_rng(hkv + budget)
    W = max(lens) + 5
    w = rows_of(kind, (len(lens), hkv, W), rng)
    ws = ws_for(len(lens), hkv)
    keep = pkc.evict_select(cuda(w), cuda(np.asarray(lens, np.int32)), budget, sinks, recent, ws)
    assert pkc.device_status(ws) == pkc.PKC_OK
    keep = keep.cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(hkv):
            np.testing.assert_array_equal(keep[b, h], select_plain(w[b, h], n, budget, sinks, recent), str((b, h)))


@pytest.mark.parametrize("m", [1, 5, 6, 8, 9, 13, 18, 19, 24])
def test_select_around_zero(m):
    """5 ordinary weights, 3 denormal ones, 10 zeros of both signs and 6
    negative ones in a shuffled row: every place the choice can end at."""
    rng = np.random.default_rng(m)
    row = np.array([3, 1, 2, 1, 0.5] + [1e-45, 3e-45, 1e-45] + [0.0, -0.0] * 5 + [-1e-45, -2, -1, -1, -3, -np.inf] + [-7],
                   np.float32)
    w = np.stack([rng.permutation(row) for _ in range(3)])[:, None]
    n = len(row)
    keep = pkc.evict_select(cuda(w), torch.full((3,), n, dtype=torch.int32, device="cuda"), m, 0, 0, ws_for(3, 1)).cpu().numpy()
    for b in range(3):
        np.testing.assert_array_equal(keep[b, 0], select_plain(w[b, 0], n, m, 0, 0))


def test_select_of_rows_longer_than_shared_memory():
    """500 rows (one block each) of 60000 weights: more than a block keeps in shared memory."""
    rng = np.random.default_rng(6)
    B, n = 500, 60000
    base = rows_of("spread", (4, n), rng)
    w = cuda(base)[torch.arange(B, device="cuda") % 4][:, None].contiguous()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    keep = pkc.evict_select(w, lens, 2000, 4, 100, ws_for(B, 1)).cpu().numpy()
    for r in range(4):
        want = select_plain(base[r], n, 2000, 4, 100)
        assert np.all(keep[r::4, 0] == want)


def test_select_of_a_request_longer_than_its_weights_is_reported():
    ws = ws_for(2, 1)
    w = torch.rand(2, 1, 64, device="cuda")
    keep = pkc.evict_select(w, torch.tensor([65, 64], dtype=torch.int32, device="cuda"), 8, 1, 1, ws)
    assert pkc.device_status(ws) == 7
    assert torch.all(keep[0] == -1)
    np.testing.assert_array_equal(keep[1, 0].cpu(), select_plain(w[1, 0].cpu().numpy(), 64, 8, 1, 1))


# ---------------------------------------------------------------------------
# Compact
# ---------------------------------------------------------------------------

def raw(c):
    """Host copies of the cache's pools (bytes)."""
    out = []
    for t in (c.k, c.v, *c.scales):
        out.append(None if t is None else t.view(torch.uint8).cpu().numpy().copy())
    return out


def compact_plain(c, pools, keep, lens, w):
    """The move on host copies; returns the weights after it."""
    w = w.copy()
    for b, n in enumerate(lens):
        budget = keep.shape[2]
        if n <= budget:
            continue
        at = lambda t: (c.bt_host[b, t // c.ps], t % c.ps)  # noqa: E731
        for h in range(c.hkv):
            for x in pools:
                if x is not None:
                    rows = [x[at(t)][h].copy() for t in keep[b, h]]
                    for j, r in enumerate(rows):
                        x[at(j)][h] = r
            w[b, h, :n] = np.concatenate([w[b, h, keep[b, h]], np.zeros(n - budget, np.float32)])
    return w


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3", "mx4"])
@pytest.mark.parametrize("hkv,ps,lens,budget", [
    (1, 16, [40, 10, 11, 9, 0], 10),
    (3, 5, [700, 699], 300),
    (8, 16, [1500, 1100, 64], 1024),
    (2, 64, [5000], 1),
    (2, 1, [130], 129),
    (1, 24, [3000], 2999),
    (2, 16, [30000, 9001], 8500),
])
def test_compact_moves_the_kept_rows_and_nothing_else(kind, hkv, ps, lens, budget):
    rng = np.random.default_rng(hkv + budget)
    c = Paged(kind, lens, hkv, ps, rng)
    B, W = len(lens), max(lens) + 7
    w = rng.random((B, hkv, W)).astype(np.float32)
    keep = np.full((B, hkv, budget), -1, np.int32)
    for b, n in enumerate(lens):
        for h in range(hkv):
            k = min(n, budget)
            keep[b, h, :k] = np.sort(rng.choice(n, k, replace=False))
    pools = raw(c)
    want_w = compact_plain(c, pools, keep, lens, w)
    dw, ws = cuda(w), ws_for(B, hkv)
    c.compact(cuda(keep), ws, dw)
    assert pkc.device_status(ws) == pkc.PKC_OK
    for got, want in zip(raw(c), pools):
        if want is not None:
            np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(dw.cpu().numpy(), want_w)
    assert c.dl.tolist() == [min(n, budget) for n in lens]
    # again, now that every request is within the budget: nothing moves
    c.compact(cuda(keep), ws, dw)
    for got, want in zip(raw(c), pools):
        if want is not None:
            np.testing.assert_array_equal(got, want)


def test_compact_leaves_requests_with_bad_pages_and_rows_with_bad_slots():
    rng = np.random.default_rng(7)
    lens, hkv, budget = [50, 60, 70], 2, 20
    c = Paged("f16", lens, hkv, 16, rng)
    keep = np.stack([np.stack([np.sort(rng.choice(n, budget, replace=False)) for _ in range(hkv)]) for n in lens]).astype(np.int32)
    keep[2, 0, 5] = keep[2, 0, 4]        # the same slot twice
    pools = raw(c)
    ok = keep.copy()
    ok[2, 0] = np.arange(budget)
    w = rng.random((3, hkv, 70)).astype(np.float32)
    w_kept = w[2, 0].copy()
    cut = [50, 0, 70]                     # request 1 has a page that is not there
    want_w = compact_plain(c, pools, ok, cut, w)
    want_w[2, 0] = w_kept
    c.bt[1, 3] = c.P + 7
    dw, ws = cuda(w), ws_for(3, hkv)
    c.compact(cuda(keep), ws, dw)
    assert pkc.device_status(ws) in (4, 7)
    for got, want in zip(raw(c), pools):
        if want is not None:
            np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(dw.cpu().numpy(), want_w)
    assert c.dl.tolist() == [20, 60, 20]
    # weights shorter than a request: that request is left as it was
    c = Paged("f16", [50, 30], 1, 16, rng)
    before = raw(c)
    keep2 = np.stack([np.arange(30, 50), np.arange(10, 30)])[:, None].astype(np.int32)
    ws, w = ws_for(2, 1), torch.rand(2, 1, 40, device="cuda")
    w0 = w.clone()
    want_w = compact_plain(c, before, keep2, [0, 30], w0.cpu().numpy())
    c.compact(cuda(keep2), ws, w)
    assert pkc.device_status(ws) == 7 and c.dl.tolist() == [50, 20]
    for got, want in zip(raw(c), before):
        if want is not None:
            np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(w.cpu().numpy(), want_w)
    # slots out of range and descending ones: nothing is read or written through them
    for bad in (-1, 1 << 30, 2 ** 31 - 1):
        c = Paged("mx4", [50], 1, 16, rng)
        before = raw(c)
        k = np.arange(30, 50, dtype=np.int32)
        k[7] = bad
        ws = ws_for(1, 1)
        c.compact(cuda(k[None, None]), ws)
        assert pkc.device_status(ws) == 7 and c.dl.tolist() == [20]
        for got, want in zip(raw(c), before):
            np.testing.assert_array_equal(got, want)


def test_compact_leaves_a_request_that_select_could_not_choose_for():
    rng = np.random.default_rng(11)
    lens, hkv, budget = [90, 40, 90, 17], 3, 16
    c = Paged("bf16", lens, hkv, 8, rng)
    w, ws = torch.rand(4, hkv, 64, device="cuda"), ws_for(4, hkv)  # requests 0 and 2 are longer than that
    c.dl[3] = 12  # within the budget; request 3 grows afterwards
    keep = pkc.evict_select(w, c.dl, budget, 2, 4, ws)
    c.dl[3] = 17
    keep[2] = torch.arange(budget, device="cuda")  # all of request 2's heads but one: the caller's own choice
    keep[2, 1, -1] = -1
    pools = raw(c)
    compact_plain(c, pools, keep.cpu().numpy(), [0, 40, 0, 0], np.zeros((4, hkv, 90), np.float32))
    ws = ws_for(4, hkv)
    c.compact(keep, ws)
    assert pkc.device_status(ws) == 7 and c.dl.tolist() == [90, 16, 90, 17]
    for got, want in zip(raw(c), pools):
        if want is not None:
            np.testing.assert_array_equal(got, want)


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
def test_serving_loop_under_a_budget(kind):
    """Decode, accumulate, and, when a request outgrows the budget, select and
    compact -- then a decode over the cut cache equals attention over the kept
    tokens, and new tokens start from weight 0."""
    rng = np.random.default_rng(11)
    hkv, g, ps, lens, budget, scale = 4, 2, 16, [90, 33, 64], 48, 0.1
    B, steps = len(lens), 3
    c = Paged(kind, lens, hkv, ps, rng, room=steps)
    W = c.bt_host.shape[1] * ps
    w, ws = torch.zeros(B, hkv, W, device="cuda"), ws_for(B, hkv * g)
    host_w = np.zeros((B, hkv, W))
    for step in range(steps):
        q = torch.from_numpy(rng.standard_normal((B, hkv * g, 128)) * 2).cuda().to(q_type(kind))
        o, lse = c.decode(q, scale, ws)
        for b, n in enumerate(c.lens):
            ro, rl, sm, vm = ref.attention(f64(q)[b], c.rows(0, b, n), c.rows(1, b, n), g, scale)
            ot, lt = ref.bounds(ro, rl, sm, vm, torch.finfo(q.dtype).eps)
            assert np.all(np.abs(f64(o)[b] - ro) <= ot + 2.0 ** -16 * vm) and np.all(np.abs(f64(lse)[b] - rl) <= lt)
        c.accumulate(q, lse, scale, w, ws, decay=0.9)
        host_w, tol = want_weights(c, q, lse, scale, host_w, 0.9, g)
        assert np.all(np.abs(f64(w) - host_w) <= (step + 1) * (tol + 2.0 ** -22))
        keep = pkc.evict_select(w, c.dl, budget, 2, 8, ws)
        hw, hk = w.cpu().numpy(), keep.cpu().numpy()
        for b, n in enumerate(c.lens):
            for h in range(hkv):
                np.testing.assert_array_equal(hk[b, h], select_plain(hw[b, h], n, budget, 2, 8))
        pools = raw(c)
        want_w = compact_plain(c, pools, hk, c.lens, hw)
        c.compact(keep, ws, w)
        for got, want in zip(raw(c), pools):
            if want is not None:
                np.testing.assert_array_equal(got, want)
        np.testing.assert_array_equal(w.cpu().numpy(), want_w)
        c.lens = [min(n, budget) for n in c.lens]
        assert c.dl.tolist() == c.lens
        host_w = want_w.astype(np.float64)
        # one new token per request, at the place the cut left free
        x = torch.from_numpy(rng.standard_normal((2, B, hkv, 128)) * 0.5).cuda()
        if c.mx4:
            pkc.append_kv_mx4(x[0].to(q_type(kind)).contiguous(), x[1].to(q_type(kind)).contiguous(),
                              torch.arange(B + 1, dtype=torch.int32, device="cuda"),
                              c.k, c.scales[0], c.v, c.scales[1], c.bt, c.dl, ws)
        else:
            y = x.float().to(E4M3).view(torch.uint8) if kind == "e4m3" else x.to(DT[kind])
            pkc.append_kv(y[0].contiguous(), y[1].contiguous(), c.k, c.v, c.bt, c.dl, ws)
        c.lens = [n + 1 for n in c.lens]
        assert c.dl.tolist() == c.lens
        for b, n in enumerate(c.lens):
            assert np.all(host_w[b, :, n - 1] == 0)
    assert pkc.device_status(ws) == pkc.PKC_OK


def test_weights_of_a_cascade_suffix_use_the_whole_row():
    """The cascade's LSE (prefix and suffix) makes the suffix's weights those
    of the whole row: what the prefix takes is missing from them."""
    rng = np.random.default_rng(12)
    hkv, g, ps, lens, L, scale = 2, 4, 16, [40, 100], 128, 0.1
    c = Paged("f16", lens, hkv, ps, rng)
    kp, vp = (torch.from_numpy(rng.standard_normal((L, hkv, 128))).cuda().half() for _ in "kv")
    q = torch.from_numpy(rng.standard_normal((2, hkv * g, 128)) * 2).cuda().half()
    ws = torch.empty(pkc.workspace_size(2, hkv * g, 0, 64), dtype=torch.uint8, device="cuda")
    pkc.workspace_init(ws)
    o, lse = pkc.cascade_decode(q, kp, vp, [0, L], [0, 2], c.k, c.v, c.bt, c.dl, scale, ws)
    w = torch.zeros(2, hkv, 112, device="cuda")
    c.accumulate(q, lse, scale, w, ws)
    got = f64(w)
    for b, n in enumerate(lens):
        for h in range(hkv):
            share = np.zeros(n)
            for i in range(h * g, h * g + g):
                keys = np.concatenate([f64(kp)[:, h], c.rows(0, b, n)[:, h]])
                s = scale * keys @ f64(q)[b, i]
                p = np.exp(s - s.max())
                share += (p / p.sum())[L:]
            # the LSE is the call's own: good to its documented 1e-3
            np.testing.assert_allclose(got[b, h, :n], share, rtol=2e-3)


def test_evictions_in_a_captured_graph_and_on_two_streams():
    """One captured step (decode, accumulate, select, compact, append) replayed,
    against the same steps uncaptured; and two workspaces at work on two
    streams at once."""
    hkv, g, ps, lens, budget, scale = 4, 4, 16, [300, 200, 256], 128, 0.1
    B = len(lens)

    def fresh():
        r = np.random.default_rng(13)
        c = Paged("bf16", lens, hkv, ps, r, room=4)
        return c, torch.zeros(B, hkv, 320, device="cuda"), ws_for(B, hkv * g)

    rng = np.random.default_rng(14)
    qs = torch.from_numpy(rng.standard_normal((3, B, hkv * g, 128))).cuda().to(torch.bfloat16)
    x = torch.from_numpy(rng.standard_normal((2, B, hkv, 128))).cuda().to(torch.bfloat16)

    def one(c, w, ws, q, keep):
        o, lse = c.decode(q, scale, ws)
        c.accumulate(q, lse, scale, w, ws, decay=0.5)
        pkc.evict_select(w, c.dl, budget, 4, 16, ws, keep=keep)
        c.compact(keep, ws, w)
        pkc.append_kv(x[0], x[1], c.k, c.v, c.bt, c.dl, ws)

    runs = []
    for mode in ("plain", "graph", "streams"):
        c, w, ws = fresh()
        keep = torch.empty(B, hkv, budget, dtype=torch.int32, device="cuda")
        q = qs[0].clone()
        if mode == "graph":
            s = torch.cuda.Stream()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                one(c, w, ws, q, keep)
            for i in range(3):
                q.copy_(qs[i])
                graph.replay()
        elif mode == "streams":
            c2, w2, ws2 = fresh()
            keep2 = torch.empty_like(keep)
            torch.cuda.synchronize()
            s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
            for i in range(3):
                for st, args in ((s1, (c, w, ws, qs[i], keep)), (s2, (c2, w2, ws2, qs[i], keep2))):
                    with torch.cuda.stream(st):
                        one(*args)
            torch.cuda.synchronize()
            assert torch.equal(w, w2) and torch.equal(c.k, c2.k) and torch.equal(keep, keep2)
        else:
            for i in range(3):
                one(c, w, ws, qs[i], keep)
        torch.cuda.synchronize()
        assert pkc.device_status(ws) == pkc.PKC_OK
        runs.append((w.clone(), keep.clone(), c.k.clone(), c.v.clone(), c.dl.tolist()))
    for r in runs[1:]:
        for a, b in zip(runs[0], r):
            assert torch.equal(a, b) if isinstance(a, torch.Tensor) else a == b
