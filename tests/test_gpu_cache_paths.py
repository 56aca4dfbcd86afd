"""The forms that the compressed, bounded cache's kernels take for batches and
long requests: several KV heads per block and page windows of the mx4 decode,
segments of many steps of the accumulated weights, rows of millions of weights
of the selection, and the mx4 cache behind a shared prefix.  References are
float64 on the GPU (numpy where whole numbers are compared)."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
import paged_kv_cascade_gb300 as pkc
from test_gpu_evict import E4M3, KINDS, q_type, rows_of, select_plain
from test_gpu_mx4 import DT, EPS, Cache, cuda, f64, table_for, ws_for

pytestmark = pytest.mark.gpu


def values(codes, scales):
    """float64 [..., 128] on the GPU of an mx4 cache's codes and scales."""
    grid = torch.tensor(np.concatenate([ref.GRID, -ref.GRID]), device=codes.device)
    nib = torch.stack((codes & 15, codes >> 4), -1)  # [..., 64 bytes, low / high]
    v = grid[nib.long()].reshape(codes.shape[:-1] + (8, 4, 4))  # [..., u, b, i]
    v = v.transpose(-3, -2).reshape(codes.shape[:-1] + (4, 32))
    f = torch.where(scales == 255, torch.nan, torch.exp2(scales.double() - 127))
    return (v * f[..., None]).reshape(codes.shape[:-1] + (128,))


def test_the_gpu_reference_is_the_numpy_one():
    rng = np.random.default_rng(1)
    codes, scales = rng.integers(0, 256, (50, 64)).astype(np.uint8), rng.integers(0, 256, (50, 4)).astype(np.uint8)
    np.testing.assert_array_equal(f64(values(cuda(codes), cuda(scales))), ref.values(codes, scales))


def mx4_pools(P, ps, hkv, seed):
    """Random codes; scales of 2^-3 .. 2 (values of about 1)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in "kv":
        out.append(torch.randint(0, 256, (P, ps, hkv, 64), generator=gen, device="cuda", dtype=torch.uint8))
        out.append(torch.randint(124, 127, (P, ps, hkv, 4), generator=gen, device="cuda", dtype=torch.uint8))
    return out


def rows(pool, table_row, n, ps):
    pages = table_row[: (n + ps - 1) // ps].clamp(min=0, max=pool.shape[0] - 1).long()
    return pool[pages].flatten(0, 1)[:n]


def check_states(q, pools, bt, lens, ps, g, scale, o, lse, dtype, missing=()):
    """The decode's states against float64 attention with mx4_reference.bounds'
    error terms; missing: (request, page number) pairs without a page."""
    eps, hkv = EPS[dtype], pools[0].shape[2]
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.all(o[b] == 0) and torch.all(lse[b] == -torch.inf)
            continue
        keys, vals = (values(rows(pools[j], bt[b], n, ps), rows(pools[j + 1], bt[b], n, ps)) for j in (0, 2))
        here = torch.ones(n, dtype=torch.bool, device="cuda")
        for r, page in missing:
            if r == b:
                here[page * ps:(page + 1) * ps] = False
        keys, vals = keys[here], vals[here]
        qd = q[b].double().reshape(hkv, g, 128)
        s = torch.einsum("hgd,thd->hgt", qd, keys) * scale
        want_l = torch.logsumexp(s, -1)
        want_o = torch.einsum("hgt,thd->hgd", torch.exp(s - want_l[..., None]), vals)
        mag = torch.einsum("hgd,thd->hgt", qd.abs(), keys.abs()).amax(-1) * scale
        vmax = vals.abs().reshape(-1, hkv, 4, 32).amax((0, 3)).repeat_interleave(32, -1)
        dp = 137 * 2.0 ** -24 * mag + 2.0 ** -20
        tol_o = (2 * dp + 2.0 ** -18)[..., None] * vmax[:, None] + want_o.abs() * eps / 2 + 2.0 ** -25
        tol_l = dp + 2.0 ** -18 + want_l.abs() * 2.0 ** -22
        off_o = (o[b].double().reshape(hkv, g, 128) - want_o).abs()
        off_l = (lse[b].double().reshape(hkv, g) - want_l).abs()
        assert torch.all(off_o <= tol_o), (b, n, (off_o / tol_o).max().item())
        assert torch.all(off_l <= tol_l), (b, n, (off_l / tol_l).max().item())


# ---------------------------------------------------------------------------
# mx4 decode: several KV heads per block, windows of pages
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("ps", [16, 8, 48])
@pytest.mark.parametrize("dtype,batch,hkv,g,longest", [
    ("f16", 640, 8, 4, 1700),   # four KV heads per block, a warp each
    ("bf16", 1250, 4, 8, 1100),
    ("bf16", 200, 8, 4, 2500),  # two heads, two warps each
    ("f16", 330, 2, 1, 2300),
    ("f16", 3, 1, 8, 9000),     # one head, four warps
])
def test_decode_forms_without_a_plan(dtype, batch, hkv, g, longest, ps):
    rng = np.random.default_rng(batch + ps)
    lens = rng.integers(0, 90, batch)
    lens[rng.choice(batch, 3, replace=False)] = [longest, longest - 17, longest // 2 + 3]
    lens = [int(x) for x in lens]
    host_bt, P = table_for(lens, ps, rng)
    # a missing page far into the longest request, one at the end of another's
    at = int(np.argmax(lens))
    missing = [(at, (longest - 100) // ps), (at, 2)]
    for r, page in missing:
        host_bt[r, page] = -1 if page == 2 else P + 5
    pools, bt, dl = mx4_pools(P, ps, hkv, batch), cuda(host_bt), cuda(np.asarray(lens, np.int32))
    q = torch.from_numpy(rng.standard_normal((batch, hkv * g, 128))).cuda().to(DT[dtype])
    ws = ws_for(batch, hkv * g)
    o, lse = pkc.paged_decode_state_mx4(q, *pools, bt, dl, 0.09, ws)
    assert pkc.device_status(ws) == 4  # PKC_ERR_BLOCK_TABLE: the missing pages
    check_states(q, pools, bt, lens, ps, g, 0.09, o, lse, dtype, missing)


@pytest.mark.parametrize("schedule", ["dynamic", "static"])
@pytest.mark.parametrize("ps", [16, 8])
@pytest.mark.parametrize("dtype,batch,hkv,g,ctas", [
    ("f16", 650, 8, 4, 304),
    ("bf16", 1300, 4, 8, 148),
    ("bf16", 180, 8, 2, 304),
    ("f16", 256, 4, 8, 40),
])
def test_decode_forms_with_a_plan(schedule, dtype, batch, hkv, g, ctas, ps):
    rng = np.random.default_rng(batch + ps)
    lens = np.minimum(np.exp(rng.normal(3.5, 1.2, batch)).astype(int), 4000)
    lens[rng.choice(batch, 3, replace=False)] = [0, 1, 5000]
    lens = [int(x) for x in lens]
    host_bt, P = table_for(lens, ps, rng)
    pools, bt, dl = mx4_pools(P, ps, hkv, batch), cuda(host_bt), cuda(np.asarray(lens, np.int32))
    q = torch.from_numpy(rng.standard_normal((batch, hkv * g, 128))).cuda().to(DT[dtype])
    ws, plan = ws_for(batch, hkv * g, ctas), pkc.plan(lens, ctas)
    pkc.plan_upload(plan, ws)
    try:
        pkc.set_decode_schedule(schedule)
        outs = [pkc.paged_decode_state_mx4(q, *pools, bt, dl, 0.09, ws, plan_buf=plan) for _ in range(3)]
    finally:
        pkc.set_decode_schedule("dynamic")
    assert pkc.device_status(ws) == pkc.PKC_OK
    check_states(q, pools, bt, lens, ps, g, 0.09, *outs[0], dtype)
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_planned_decodes_of_two_graphs_over_one_workspace():
    """Decode and weights captured twice with one workspace and plan, replayed
    in turn with other queries: the same bits as without a graph."""
    rng = np.random.default_rng(9)
    lens, hkv, g, ps, ctas = [3000, 17, 0, 900, 64], 4, 8, 16, 148
    B = len(lens)
    host_bt, P = table_for(lens, ps, rng)
    pools, bt, dl = mx4_pools(P, ps, hkv, 1), cuda(host_bt), cuda(np.asarray(lens, np.int32))
    qs = torch.from_numpy(rng.standard_normal((6, B, hkv * g, 128))).cuda().bfloat16()
    ws, plan = ws_for(B, hkv * g, ctas), pkc.plan(lens, ctas)
    pkc.plan_upload(plan, ws)

    def one(q, w, o=None, lse=None):
        o, lse = pkc.paged_decode_state_mx4(q, *pools, bt, dl, 0.1, ws, plan_buf=plan, o=o, lse=lse)
        pkc.accumulate_weights(q, lse, pools[0], bt, dl, 0.1, w, ws, k_scales=pools[1], decay=0.0)
        return o, lse, w

    want = [one(q, torch.zeros(B, hkv, 3008, device="cuda")) for q in qs]
    check_states(qs[0], pools, bt, lens, ps, g, 0.1, *want[0][:2], "bf16")
    graphs, stream = [], torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        bufs = (qs[0].clone(), torch.zeros(B, hkv, 3008, device="cuda"), torch.empty_like(qs[0]),
                torch.empty(qs.shape[1:3], device="cuda"))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            one(*bufs)
        graphs.append((graph, bufs))
    for i, q in enumerate(qs):
        graph, (gq, w, o, lse) = graphs[i % 2]
        gq.copy_(q)
        graph.replay()
        for got, ref_ in zip((o, lse, w), want[i]):
            assert torch.equal(got, ref_)
    assert pkc.device_status(ws) == pkc.PKC_OK


def test_calls_without_requests_or_rows():
    """A batch of none, and no new rows: nothing is launched, nothing changes."""
    u8, i32 = torch.uint8, torch.int32
    z = lambda *s, d=u8: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    pools = [torch.full((2, 16, 2, n), 7, dtype=u8, device="cuda") for n in (64, 4, 64, 4)]
    ws = ws_for(1, 2)
    for B in (0, 1):
        bt, lens, ip = z(B, 3, d=i32), z(B, d=i32), z(B + 1, d=i32)
        x = z(0, 2, 128, d=torch.float16)
        pkc.append_kv_mx4(x, x, ip, *pools, bt, lens, ws)
        k, v = pkc.gather_kv_mx4(*pools, bt, lens, ip, 0, ws)
        assert k.shape == v.shape == (0, 2, 128)
        q = z(B, 2, 128, d=torch.float16)
        o, lse = pkc.paged_decode_state_mx4(q, *pools, bt, lens, 0.1, ws)
        assert torch.all(o == 0) and torch.all(lse == -torch.inf) and o.shape == q.shape
        w = torch.ones(B, 2, 48, device="cuda")
        pkc.accumulate_weights(q, lse, pools[0], bt, lens, 0.1, w, ws, k_scales=pools[1])
        keep = pkc.evict_select(w, lens, 5, 1, 2, ws)
        assert keep.shape == (B, 2, 5) and torch.all(keep == -1)
        pkc.evict_compact(keep, pools[0], pools[2], bt, lens, ws, weights=w, k_scales=pools[1], v_scales=pools[3])
        assert torch.all(w == 1) and torch.all(lens == 0)
    assert all(torch.all(p == 7) for p in pools) and pkc.device_status(ws) == pkc.PKC_OK


# ---------------------------------------------------------------------------
# Accumulated weights: segments of many steps
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("batch,hkv,g,ps,longest", [
    (128, 8, 4, 16, 2400),   # a head per warp, 16 or (mx4) 32 steps a segment
    (128, 8, 2, 5, 2400),
    (160, 2, 8, 48, 2500),   # two warps per head
    (160, 1, 1, 16, 3000),   # four
    (160, 1, 8, 7, 3000),
])
def test_weights_of_segments_of_many_steps(kind, batch, hkv, g, ps, longest):
    rng = np.random.default_rng(batch + ps)
    lens = np.minimum(np.exp(rng.normal(5.5, 1.2, batch)).astype(int), longest)
    lens[rng.choice(batch, 8, replace=False)] = [0, 1, longest, longest - 1, 257, 511, 513, 1025]
    lens = [int(x) for x in lens]
    host_bt, P = table_for(lens, ps, rng)
    at = int(np.argmax(lens))
    missing = [(at, 9), (at, (longest - 40) // ps)]
    for r, page in missing:
        host_bt[r, page] = -3
    bt, dl = cuda(host_bt), cuda(np.asarray(lens, np.int32))
    gen = torch.Generator(device="cuda").manual_seed(ps)
    k_scale, scales = 1.0, None
    if kind.startswith("mx4"):
        k, scales = mx4_pools(P, ps, hkv, batch)[:2]
    else:
        k = torch.randn((P, ps, hkv, 128), generator=gen, device="cuda").to(E4M3 if kind == "e4m3" else DT[kind])
        if kind == "e4m3":
            k, k_scale = k.view(torch.uint8), 0.5
    q = torch.from_numpy(rng.standard_normal((batch, hkv * g, 128))).cuda().to(q_type(kind))
    lse = torch.from_numpy(rng.normal(2.0, 1.0, (batch, hkv * g))).float().cuda()
    W = host_bt.shape[1] * ps
    w0 = torch.rand((batch, hkv, W), generator=gen, device="cuda")
    ws, scale, decay = ws_for(batch, hkv * g), 0.09, 0.75
    w = w0.clone()
    pkc.accumulate_weights(q, lse, k, bt, dl, scale, w, ws, decay=decay, k_scale=k_scale, k_scales=scales)
    assert pkc.device_status(ws) == 4
    for b, n in enumerate(lens):
        assert torch.equal(w[b, :, n:], w0[b, :, n:])  # nothing behind the length
        x = rows(k, bt[b], n, ps)
        keys = values(x, rows(scales, bt[b], n, ps)) if scales is not None else \
            x.view(E4M3).double() * k_scale if kind == "e4m3" else x.double()
        qd, ld = q[b].double().reshape(hkv, g, 128), lse[b].double().reshape(hkv, g, 1)
        p = torch.exp(torch.einsum("hgd,thd->hgt", qd, keys) * scale - ld)
        mag = torch.einsum("hgd,thd->hgt", qd.abs(), keys.abs()) * scale
        old = w0[b, :, :n].double()
        want = decay * old + p.sum(1)
        # as in test_gpu_evict.want_weights
        err = (p * (137 * 2.0 ** -24 * mag + ld.abs() * 2.0 ** -22 + 2.0 ** -21)).sum(1)
        tol = 1.01 * err + 2.0 ** -22 * want + 2.0 ** -126
        for r, page in missing:
            if r == b:
                want[:, page * ps:(page + 1) * ps] = old[:, page * ps:(page + 1) * ps]
        off = (w[b, :, :n].double() - want).abs()
        assert torch.all(off <= tol), (b, n, (off / tol).max().item() if n else 0)


# ---------------------------------------------------------------------------
# Select: rows of up to 2^22 weights
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["spread", "equal", "few values", "mostly zero", "odd values"])
@pytest.mark.parametrize("n,W,budget,sinks,recent", [
    (300001, 300005, 20000, 4, 1000),       # a cluster per row, keys not held
    (4100003, 1 << 22, 200001, 0, 33),
])
def test_select_of_rows_that_no_cluster_holds(kind, n, W, budget, sinks, recent):
    rng = np.random.default_rng(n)
    w = rows_of(kind, (1, 1, W), rng)
    ws = ws_for(1, 1)
    keep = pkc.evict_select(cuda(w), torch.full((1,), n, dtype=torch.int32, device="cuda"), budget, sinks, recent, ws)
    assert pkc.device_status(ws) == pkc.PKC_OK
    np.testing.assert_array_equal(keep[0, 0].cpu().numpy(), select_plain(w[0, 0], n, budget, sinks, recent))


def test_select_of_short_requests_in_a_wide_buffer():
    """160 rows of 2^19 + 100 weights (two blocks a row for their width), of
    which a request uses few: the second block has none, or all rows have some."""
    rng = np.random.default_rng(5)
    B, W, budget = 160, (1 << 19) + 100, 50
    w = torch.zeros(B, 1, W, device="cuda")
    lens = rng.integers(0, 3000, B)
    lens[:4] = [51, 52, 60, 83]
    lens[4] = W
    host = [rows_of("mostly zero" if b % 2 else "spread", (int(n),), rng) for b, n in enumerate(lens)]
    for b, x in enumerate(host):
        w[b, 0, :len(x)] = cuda(x)
    ws = ws_for(B, 1)
    keep = pkc.evict_select(w, cuda(lens.astype(np.int32)), budget, 1, 7, ws).cpu().numpy()
    assert pkc.device_status(ws) == pkc.PKC_OK
    for b, x in enumerate(host):
        np.testing.assert_array_equal(keep[b, 0], select_plain(x, len(x), budget, 1, 7), str(b))


# ---------------------------------------------------------------------------
# An mx4 cache behind a shared prefix
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("planned", [False, True])
def test_mx4_cache_behind_a_shared_prefix(dtype, planned):
    """The prefix's float32 state and the mx4 cache's state merged: attention
    over both; and the weights from the merged LSE are those of the whole row."""
    rng = np.random.default_rng(6)
    hkv, g, ps, lens, L, scale, ctas = 2, 4, 16, [40, 0, 700], 256, 0.1, 16
    B = len(lens)
    c = Cache(lens, hkv, ps, rng)
    d, bt, dl = c.device()
    kp, vp = (torch.from_numpy(rng.standard_normal((L, hkv, 128))).cuda().to(DT[dtype]) for _ in "kv")
    q = torch.from_numpy(rng.standard_normal((B, hkv * g, 128)) * 2).cuda().to(DT[dtype])
    ws = torch.empty(pkc.workspace_size(B, hkv * g, ctas, 64), dtype=torch.uint8, device="cuda")
    pkc.workspace_init(ws)
    plan = pkc.plan(lens, ctas) if planned else None
    if planned:
        pkc.plan_upload(plan, ws)
    po, pl = pkc.prefix_attention_state(q, kp, vp, [0, L], [0, B], scale, ws)
    so, sl = pkc.paged_decode_state_mx4(q, *d, bt, dl, scale, ws, plan_buf=plan)
    o, lse = pkc.merge_states_to(torch.stack((po, so.float()), 1), torch.stack((pl, sl), 1), q.dtype)
    w = torch.zeros(B, hkv, 704, device="cuda")
    pkc.accumulate_weights(q, lse, d[0], bt, dl, scale, w, ws, k_scales=d[1])
    assert pkc.device_status(ws) == pkc.PKC_OK
    got_o, got_l, got_w = f64(o), f64(lse), f64(w)
    for b, n in enumerate(lens):
        k, v = (np.concatenate([f64(x), y[b]]) for x, y in ((kp, c.k), (vp, c.v)))
        ro, rl, _, vm = ref.attention(f64(q)[b], k, v, g, scale)
        # the prefix and the merge are good to the library's documented 2e-3 and
        # 1e-3; the cache's part is rounded to 16 bits before the merge, the
        # result after it
        assert np.all(np.abs(got_o[b] - ro) <= 2e-3 + EPS[dtype] / 2 * (vm + np.abs(ro)))
        assert np.all(np.abs(got_l[b] - rl) <= 1e-3)
        for h in range(hkv):
            share = np.zeros(n)
            for i in range(h * g, h * g + g):
                s = scale * (k[:, h] @ f64(q)[b, i])
                share += np.exp(s - rl[i])[L:]
            np.testing.assert_allclose(got_w[b, h, :n], share, rtol=2e-3)
            assert np.all(got_w[b, h, n:] == 0)
