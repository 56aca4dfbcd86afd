"""Prompts, chunks and single tokens through the calls as they are used together:
pages, rotary append, chunk attention, and the decode, eviction, prefix and merge
calls around them, each against its definition in 64 bits over what the pool holds."""
import math

import pytest
import torch

import paged_kv_cascade_gb300 as pkc
import prompt_reference as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
I32 = torch.int32
SCALE = 1 / math.sqrt(128)


def e4m3_values():
    return torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()


def dev(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Server:
    """The state that a server keeps, on the device, and its plain twin."""

    def __init__(self, batch, hq, hkv, dtype, page, num_pages, stride, seed, codes=False):
        self.batch, self.hq, self.hkv, self.dtype, self.page, self.num_pages = batch, hq, hkv, dtype, page, num_pages
        self.gen = torch.Generator().manual_seed(seed)
        self.table = torch.full((batch, stride), -1, dtype=I32, device="cuda")
        self.lens = torch.zeros(batch, dtype=I32, device="cuda")
        self.free = pkc.page_pool(num_pages)
        shape = (num_pages, page, hkv, 128)
        self.k, self.v = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") if codes else
                          torch.full(shape, math.nan, dtype=dtype, device="cuda") for _ in "kv")
        self.freq, self.amp = pkc.rope_frequencies(128)
        self.ws = torch.empty(pkc.workspace_size(batch, hq) + pkc.chunk_workspace_size(), dtype=torch.uint8, device="cuda")
        pkc.workspace_init(self.ws)
        self.h_table, self.h_lens, self.h_free = [[-1] * stride for _ in range(batch)], [0] * batch, set(range(num_pages))
        self.keys = {}  # slot -> (key before the turn, position, value)

    def tokens(self, n):
        return torch.randn((n, self.hq + 2 * self.hkv, 128), generator=self.gen).to(self.dtype)

    def append(self, new, k_scale=1.0, v_scale=1.0):
        """Pages and rows of new[b] tokens per request; the turned queries and the row ranges."""
        indptr = [0]
        for n in new:
            indptr.append(indptr[-1] + n)
        qkv = self.tokens(indptr[-1])
        d = qkv.cuda()
        slots, pos, _ = pkc.assign_pages(self.table, self.lens, dev(indptr), indptr[-1], self.free, self.page, self.num_pages, self.ws,
                                         seqlens_out=self.lens)
        h_slots, h_pos, self.h_lens, status = ref.assign(self.h_table, self.h_lens, indptr, indptr[-1], self.h_free, self.page)
        assert status == 0 and slots.tolist() == h_slots and pos.tolist() == h_pos
        assert self.table.tolist() == self.h_table and self.lens.tolist() == self.h_lens
        assert pkc.device_status(self.ws) == 0
        a, b = self.hq, self.hq + self.hkv
        q = pkc.rope_append_kv(d[:, :a], d[:, a:b], d[:, b:], pos, slots, self.freq, self.k, self.v, self.ws, amplitude=self.amp,
                               k_scale=k_scale, v_scale=v_scale)
        for i, s in enumerate(h_slots):
            self.keys[s] = (qkv[i, a:b], h_pos[i], qkv[i, b:])
        want, size = ref.rotate(qkv[:, :a], torch.tensor(h_pos), self.freq.cpu(), False, self.amp)
        self.near(q.cpu(), want, size)
        return q, dev(indptr), indptr

    def near(self, got, want, size):
        """A turned row: 2^-19 of its terms for the angle, sine, cosine and sum (see the rotary tests), half a step."""
        off = (got.double() - want).abs() - (ref.HALF_STEP[self.dtype] * want.abs() + 2.0 ** -19 * size + 2.0 ** -25)
        assert off.numel() == 0 or float(off.max()) <= 0

    def check_pool(self):
        """Every cached row: the key turned by its position, the value as it was."""
        slots = sorted(self.keys)
        raw = torch.stack([self.keys[s][0] for s in slots])
        want, size = ref.rotate(raw, torch.tensor([self.keys[s][1] for s in slots]), self.freq.cpu(), False, self.amp)
        self.near(self.k.cpu().reshape(-1, self.hkv, 128)[slots], want, size)
        assert torch.equal(self.v.cpu().reshape(-1, self.hkv, 128)[slots], torch.stack([self.keys[s][2] for s in slots]))

    def reference(self, q, indptr, window=0):
        return ref.chunk(q.cpu(), indptr, self.k.cpu(), self.v.cpu(), self.table.cpu(), self.h_lens, SCALE, True, window)

    def chunk(self, q, d_indptr, indptr, window=0):
        o, lse = pkc.paged_chunk_state(q, d_indptr, self.k, self.v, self.table, self.lens, SCALE, self.ws, window=window)
        ref.check_chunk(o, lse, self.reference(q, indptr, window), self.dtype)
        assert pkc.device_status(self.ws) == 0
        return o, lse

    def release(self):
        pkc.release_pages(self.table, self.lens, self.free, self.page, self.num_pages, self.ws)
        ref.release(self.h_table, self.h_lens, self.h_free, self.page)
        assert self.table.tolist() == self.h_table and ref.pool_set(self.free, self.num_pages) == self.h_free
        assert pkc.device_status(self.ws) == 0


@pytest.mark.parametrize("hq,hkv,dtype,page", [(4, 4, F16, 16), (8, 1, BF16, 5), (4, 2, BF16, 64)])
def test_prompts_steps_evictions_and_new_requests(hq, hkv, dtype, page):
    s = Server(4, hq, hkv, dtype, page, num_pages=-(-1200 // page), stride=-(-500 // page), seed=hq)
    # prompts, then further chunks beside single tokens
    for new in ([200, 0, 37, 130], [64, 1, 1, 0], [1, 1, 5, 1], [130, 3, 0, 17]):
        s.chunk(*s.append(new))
    s.check_pool()
    # one token each: the decode call and the chunk call see the same states
    q, d_indptr, indptr = s.append([1, 1, 1, 1])
    o, lse = s.chunk(q, d_indptr, indptr)
    od, lsed = pkc.paged_decode_state(q, s.k, s.v, s.table, s.lens, SCALE, s.ws)
    want = s.reference(q, indptr)
    assert torch.all((lsed.double().cpu() - want[1]).abs() <= want[3] + 2.0 ** -23 * want[1].abs())
    assert float(((od - o).abs().double().cpu() - 2 * (want[2] + 2 * ref.HALF_STEP[dtype] * (want[0].abs() + want[2]))).max()) <= 2.0 ** -24
    s.chunk(*s.append([3, 3, 3, 3]), window=50)
    # a budget: the kept tokens move to the front, the pages behind them go back to the pool
    weights = torch.zeros((4, hkv, int(s.table.shape[1]) * page), device="cuda")
    q, d_indptr, indptr = s.append([1, 1, 1, 1])
    o, lse = s.chunk(q, d_indptr, indptr)
    pkc.accumulate_weights(q, lse, s.k, s.table, s.lens, SCALE, weights, s.ws)
    keep = pkc.evict_select(weights, s.lens, 60, 4, 20, s.ws)
    pkc.evict_compact(keep, s.k, s.v, s.table, s.lens, s.ws, weights=weights)
    s.h_lens = [min(n, 60) for n in s.h_lens]
    assert s.lens.tolist() == s.h_lens
    free = len(s.h_free)
    s.release()
    assert len(s.h_free) > free
    s.chunk(*s.append([100, 1, 30, 2]))
    # a request ends, another takes its place and its pages
    s.lens[2] = 0
    s.h_lens[2] = 0
    s.release()
    s.chunk(*s.append([1, 1, 210, 1]))
    s.lens.zero_()
    s.h_lens = [0] * 4
    s.release()
    assert len(s.h_free) == s.num_pages


def test_a_captured_step_replayed():
    """Pages, rotary append and chunk attention of two tokens a request as one graph, replayed over a growing cache
    while a second state's eager calls run on another stream."""
    a, b = (Server(3, 4, 2, BF16, 16, 60, 12, seed=9) for _ in range(2))
    for s in (a, b):
        s.chunk(*s.append([50, 3, 16]))
    qkv = torch.empty((6, 8, 128), dtype=BF16, device="cuda")
    indptr = dev([0, 2, 4, 6])
    slots = torch.empty(6, dtype=torch.int64, device="cuda")
    pos = torch.empty(6, dtype=I32, device="cuda")
    o, lse, qt = torch.empty((6, 4, 128), dtype=BF16, device="cuda"), torch.empty((6, 4), device="cuda"), torch.empty((6, 4, 128), dtype=BF16, device="cuda")

    def step(s, qkv, slots, pos, qt, o, lse):
        pkc.assign_pages(s.table, s.lens, indptr, 6, s.free, 16, 60, s.ws, slots=slots, positions=pos, seqlens_out=s.lens)
        pkc.rope_append_kv(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], pos, slots, s.freq, s.k, s.v, s.ws, q_out=qt)
        pkc.paged_chunk_state(qt, indptr, s.k, s.v, s.table, s.lens, SCALE, s.ws, o=o, lse=lse)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph):
        step(a, qkv, slots, pos, qt, o, lse)
    for i in range(12):
        x = a.tokens(6).cuda()
        qkv.copy_(x)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = torch.empty_like(qt), torch.empty_like(o), torch.empty_like(lse)
            step(b, x, torch.empty_like(slots), torch.empty_like(pos), *got)
        graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        for u, v in zip((qt, o, lse), got):
            assert torch.equal(u, v)
        for u, v in ((a.table, b.table), (a.lens, b.lens), (a.free, b.free)):
            assert torch.equal(u, v)
    assert a.lens.tolist() == [74, 27, 40]
    a.h_lens = a.lens.tolist()
    ref.check_chunk(o, lse, ref.chunk(qt.cpu(), [0, 2, 4, 6], a.k.cpu(), a.v.cpu(), a.table.cpu(), a.h_lens, SCALE), BF16)
    assert pkc.device_status(a.ws) == 0 and pkc.device_status(b.ws) == 0


def test_codes_for_the_fp8_decode():
    """Prompts appended as e4m3 codes, read by the fp8 decode: its states over the values that the codes stand for."""
    s = Server(3, 8, 2, F16, 16, 40, 12, seed=3, codes=True)
    ks, vs = 0.03125, 0.0625
    s.append([100, 20, 1], ks, vs)
    q, _, indptr = s.append([1, 1, 1], ks, vs)
    o, lse = pkc.paged_decode_state_fp8(q, s.k, s.v, s.table, s.lens, SCALE, s.ws, k_scale=ks, v_scale=vs)
    k, v = (e4m3_values()[x.cpu().long()] * f for x, f in ((s.k, ks), (s.v, vs)))
    want = ref.chunk(q.cpu(), indptr, k, v, s.table.cpu(), s.h_lens, SCALE)
    ref.check_chunk(o, lse, want, F16)
    # (what the codes stand for is near the turned keys: half an e4m3 step, 2^-4 of the value, and the smallest step)
    for slot, (key, at, value) in s.keys.items():
        turned, _ = ref.rotate(key[None], torch.tensor([at]), s.freq.cpu(), False, s.amp)
        got = k.reshape(-1, 2, 128)[slot], v.reshape(-1, 2, 128)[slot]
        for x, y, f in zip(got, (turned[0], value.double()), (ks, vs)):
            assert float(((x - y).abs() - (2.0 ** -4 + 2.0 ** -10) * y.abs()).max()) <= f * 2.0 ** -9


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_chunk_behind_a_shared_prefix(dtype):
    """New tokens of several requests behind one prefix: the prefix call with a row per token, the chunk call's
    float32 states, and the merge of the two."""
    L = 300
    s = Server(3, 8, 2, dtype, 16, 60, 12, seed=5)
    kp, vp = (torch.randn((L, 2, 128), generator=s.gen).to(dtype) for _ in "kv")
    s.append([20, 0, 100])
    q, d_indptr, indptr = s.append([40, 1, 7])
    T = indptr[-1]
    ws = torch.empty(pkc.workspace_size(T, 8, 0, 64), dtype=torch.uint8, device="cuda")
    pkc.workspace_init(ws)
    po, pl = pkc.prefix_attention_state(q, kp.cuda(), vp.cuda(), [0, L], [0, T], SCALE, ws)
    so, sl = pkc.paged_chunk_state(q, d_indptr, s.k, s.v, s.table, s.lens, SCALE, s.ws, out_dtype=torch.float32)
    o, lse = pkc.merge_states_to(torch.stack((po, so), 1), torch.stack((pl, sl), 1), dtype)
    # the same rows over a cache that begins with the prefix
    lens = [n + L for n in s.h_lens]
    k, v = (torch.zeros((3, max(lens), 2, 128), dtype=dtype) for _ in "kv")
    for b, n in enumerate(s.h_lens):
        pages = s.table[b].cpu()[:-(-n // 16)].long()
        for x, pre, pool in ((k, kp, s.k), (v, vp, s.v)):
            x[b, :L] = pre
            x[b, L:L + n] = pool.cpu()[pages].reshape(-1, 2, 128)[:n]
    want = ref.chunk(q.cpu(), indptr, k, v, torch.arange(3)[:, None], lens, SCALE)
    # two states' errors instead of one's, and four float32 roundings where they are merged
    want = want[0], want[1], 2 * want[2] + 2.0 ** -21, 2 * want[3] + 2.0 ** -21
    ref.check_chunk(o, lse, want, dtype)
    assert pkc.device_status(ws) == 0 and pkc.device_status(s.ws) == 0


def test_a_pool_past_32_bits():
    """Pages whose rows lie more than 2^32 elements into the pool."""
    page, hkv, num_pages = 16, 16, 140_000  # 4.6 G elements a pool
    k, v = (torch.empty((num_pages, page, hkv, 128), dtype=BF16, device="cuda") for _ in "kv")
    gen = torch.Generator().manual_seed(6)
    lens, free = [70, 0, 33], set(range(num_pages - 12, num_pages)) - {num_pages - 3}
    table = [[num_pages - 20 - j for j in range(5)] + [-1] * 15, [-1] * 20, [num_pages - 30, 3, num_pages - 31] + [-1] * 17]
    past = torch.randn((2, 3, 80, hkv, 128), generator=gen).to(BF16)
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            k[table[b][j]], v[table[b][j]] = (x[b, j * page:(j + 1) * page].cuda() for x in past)
    ws = torch.empty(pkc.chunk_workspace_size(), dtype=torch.uint8, device="cuda")
    pkc.workspace_init(ws)
    indptr = [0, 40, 47, 60]
    d_table, d_free, d_lens = dev(table), ref.pool_words(free, num_pages).cuda(), dev(lens)
    slots, pos, _ = pkc.assign_pages(d_table, d_lens, dev(indptr), 60, d_free, page, num_pages, ws, seqlens_out=d_lens)
    h_slots, h_pos, h_lens, status = ref.assign(table, lens, indptr, 60, free, page)
    assert status == 0 and slots.tolist() == h_slots and pos.tolist() == h_pos and d_lens.tolist() == h_lens and d_table.tolist() == table
    freq, _ = pkc.rope_frequencies(128)
    qkv = torch.randn((60, 3 * hkv, 128), generator=gen).to(BF16)
    d = qkv.cuda()
    q = pkc.rope_append_kv(d[:, :hkv], d[:, hkv:2 * hkv], d[:, 2 * hkv:], pos, slots, freq, k, v, ws)
    rows = v.view(-1, hkv, 128)[slots]
    assert torch.equal(rows.cpu(), qkv[:, 2 * hkv:])
    o, lse = pkc.paged_chunk_state(q, dev(indptr), k, v, d_table, d_lens, SCALE, ws)
    # the same tokens in a small pool
    small = sorted({p for r in table for p in r if p >= 0})
    near = [[small.index(p) if p >= 0 else -1 for p in r] for r in table]
    at = torch.tensor(small, device="cuda")
    ref.check_chunk(o, lse, ref.chunk(q.cpu(), indptr, k[at].cpu(), v[at].cpu(), torch.tensor(near), h_lens, SCALE), BF16)
    pkc.release_pages(d_table, torch.zeros_like(d_lens), d_free, page, num_pages, ws)
    ref.release(table, [0, 0, 0], free, page)
    assert ref.pool_set(d_free, num_pages) == free and d_table.tolist() == table
    assert pkc.device_status(ws) == 0
