"""Attention of a chunk of new tokens over the paged cache, against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cascade_gb300 as pkc
import prompt_reference as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
I32 = torch.int32


def workspace(extra=0):
    ws = torch.empty(pkc.chunk_workspace_size() + extra, dtype=torch.uint8, device="cuda")
    pkc.workspace_init(ws)
    return ws


class Case:
    """Requests of (new, past) tokens; unused slots, pages and table entries are poison."""

    def __init__(self, reqs, hq, hkv, dtype, page=16, seed=0, lead=0, trail=0, scale=None, sharp=1.0):
        rng = np.random.default_rng(seed)
        self.lens = [n + past for n, past in reqs]
        self.indptr = np.cumsum([lead] + [n for n, _ in reqs]).tolist()
        self.total = self.indptr[-1] + trail
        need = [-(-max(n, 0) // page) for n in self.lens]
        pages = sum(need) + 3
        perm = rng.permutation(pages).tolist()
        width = max(max(need), 1) + 1
        table = torch.full((len(reqs), width), -1, dtype=I32)
        gen = torch.Generator().manual_seed(seed)
        self.k = torch.full((pages, page, hkv, 128), math.nan, dtype=dtype)
        self.v = torch.full((pages, page, hkv, 128), math.nan, dtype=dtype)
        for b, n in enumerate(self.lens):
            for j in range(need[b]):
                p = perm.pop()
                table[b, j] = p
                m = min(page, n - j * page)
                self.k[p, :m] = torch.randn((m, hkv, 128), generator=gen).to(dtype)
                self.v[p, :m] = torch.randn((m, hkv, 128), generator=gen).to(dtype)
        self.q = (sharp * torch.randn((self.total, hq, 128), generator=gen)).to(dtype)
        self.table, self.dtype, self.hq = table, dtype, hq
        self.scale = 1 / math.sqrt(128) if scale is None else scale
        self.ws = workspace()

    def run(self, causal=True, window=0, **more):
        more.setdefault("o", torch.full(self.q.shape, 7.0, dtype=more.pop("out_dtype", self.dtype), device="cuda"))
        more.setdefault("lse", torch.full(self.q.shape[:2], 7.0, device="cuda"))
        return pkc.paged_chunk_state(self.q.cuda(), torch.tensor(self.indptr, dtype=I32, device="cuda"), self.k.cuda(), self.v.cuda(), self.table.cuda(),
                                     torch.tensor(self.lens, dtype=I32, device="cuda"), self.scale, self.ws, causal=causal, window=window, **more)

    def reference(self, causal=True, window=0):
        return ref.chunk(self.q, self.indptr, self.k, self.v, self.table, self.lens, self.scale, causal, window)

    def check(self, causal=True, window=0, status=0, **more):
        o, lse = self.run(causal, window, **more)
        rows = slice(self.indptr[0], self.indptr[-1])
        ref.check_chunk(o, lse, self.reference(causal, window), o.dtype, rows)
        for x in (o, lse):  # rows of no request as they were
            assert (x[:self.indptr[0]] == 7).all() and (x[self.indptr[-1]:] == 7).all()
        assert pkc.device_status(self.ws) == status
        return o, lse


REQS = {
    "one": [(1, 0)], "single": [(1, 300)], "small": [(3, 40), (1, 0), (2, 127), (4, 128)], "prompt": [(200, 0)],
    "edges": [(128, 0), (127, 1), (129, 128), (64, 192)], "ragged": [(0, 50), (37, 91), (1, 513), (0, 0), (150, 3), (65, 64)],
    "tall": [(300, 77)], "long": [(5, 3001)],
}


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (4, 1), (8, 1)])
@pytest.mark.parametrize("reqs", list(REQS))
def test_states(reqs, hq, hkv, dtype):
    Case(REQS[reqs], hq, hkv, dtype, seed=hq).check()


@pytest.mark.parametrize("page", [1, 2, 4, 5, 8, 20, 24, 32, 48, 64, 128, 256, 1000])
def test_page_sizes(page):
    Case([(70, 60), (1, 259), (33, 0)], 4, 2, BF16, page=page, seed=page).check()


@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 1)])
@pytest.mark.parametrize("window", [1, 2, 16, 100, 127, 128, 129, 300])
def test_windows(window, hq, hkv):
    Case([(150, 200), (1, 400), (90, 0), (3, 17)], hq, hkv, F16, seed=window).check(window=window)


@pytest.mark.parametrize("window", [0, 50])
def test_not_causal(window):
    Case([(60, 100), (1, 30), (140, 0)], 4, 1, BF16, seed=3).check(causal=False, window=window)


def test_rows_before_the_first_token():
    """More rows than cached tokens: the first ones attend to nothing."""
    c = Case([(40, -15), (3, -3), (130, -128), (5, 9)], 2, 1, F16, seed=4)
    c.check()
    c.check(window=3)
    c.check(causal=False)


def test_float32_states_and_rows_of_no_request():
    c = Case([(30, 100), (200, 10)], 4, 1, BF16, lead=5, trail=9, seed=5)
    o, lse = c.check(out_dtype=torch.float32)
    assert o.dtype == torch.float32
    o16, lse16 = c.check()
    assert torch.equal(lse, lse16) and torch.equal(o[5:-9].bfloat16(), o16[5:-9])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_sharp_and_flat_scores(dtype):
    Case([(80, 200)], 4, 1, dtype, seed=6, sharp=12.0).check()
    Case([(80, 200)], 4, 1, dtype, seed=6, scale=0.0).check()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1)])
def test_later_tokens_have_no_influence(hq, hkv, bad):
    """A key and a value that a row does not attend to may hold anything."""
    c = Case([(140, 30)], hq, hkv, F16, seed=8)
    want = c.reference()
    for t in (100, 168):
        page, slot = int(c.table[0, t // 16]), t % 16
        c.v[page, slot, 0, 5] = bad
        c.k[page, slot, 0] = bad
    o, lse = c.run()
    assert pkc.device_status(c.ws) == 0
    ref.check_chunk(o, lse, want, F16, slice(0, 70))  # rows 0 .. 69 stand at positions 30 .. 99
    later = o[70:].cpu()
    assert not torch.isfinite(later[:, :, 5]).any()
    o, lse = c.run(window=60)
    mask = [i for i in range(140) if not (30 + i >= 100 and 30 + i - 60 < 100) and not (30 + i >= 168)]
    want = ref.chunk(c.q, c.indptr, torch.nan_to_num(c.k, 0, 0, 0), torch.nan_to_num(c.v, 0, 0, 0), c.table, c.lens, c.scale, True, 60)
    ref.check_chunk(o, lse, want, F16, mask)


@pytest.mark.parametrize("dtype,q_exp,k_exp", [(F16, 2, 8), (F16, 14, 8), (BF16, 14, 8), (BF16, 30, 40)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_far_out(dtype, q_exp, k_exp, sign):
    """Scores of 2^16 to 2^77, where a float32 holds no fraction, or no units, of the
    exponent: the largest one's value comes out, or the mean of those that share it.

    q holds a power of two in dim 0 and zeros, so a score is its key's dim 0 times
    that power, exactly, and two different ones lie more than 2^9 apart (weights
    exp(-2^9) = 0 in 32 bits).  The rows that share the largest one share its weight
    too, which need not be 1: it is exp2 of what is lost where scale q.k log2(e) is
    rounded, so it is rounded to 16 bits where it meets V, half a step, and O is
    rounded, another half.
    The values are below 2^3 and sum in 32 bits: 2^-19 for a few roundings.  LSE has
    the rounding of the scaled score and of the sum's logarithm."""
    c = Case([(150, 700), (3, 200), (1, 0), (140, 0)], 4, 1, dtype, seed=11, scale=1.0)
    gen = torch.Generator().manual_seed(12)
    c.q[:] = 0
    c.q[..., 0] = 2.0 ** q_exp
    rank = torch.randint(1, 100, c.k.shape[:3], generator=gen)
    c.k[..., 0] = torch.where(c.k[..., 0].isnan(), c.k[..., 0], (sign * rank * 2.0 ** k_exp).to(dtype))
    o, lse = c.run()
    assert pkc.device_status(c.ws) == 0
    want, want_lse, _, _ = c.reference()
    assert float(((o.double().cpu() - want).abs() - 2 * ref.HALF_STEP[dtype] * want.abs()).max()) <= 2.0 ** -19
    assert torch.all((lse.double().cpu() - want_lse).abs() <= 2.0 ** -21 * want_lse.abs())


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_value_that_is_not_finite(bad):
    """Only V is bad: the scores are ordinary, and O is what the sum gives in that element alone."""
    c = Case([(150, 200)], 4, 2, BF16, seed=9)
    want = c.reference()
    page, slot = int(c.table[0, 300 // 16]), 300 % 16
    c.v[page, slot, 1, 17] = bad
    o, lse = c.run()
    o = o.cpu()
    hit = o[100:, 2:, 17]
    assert hit.isnan().all() if math.isnan(bad) else (hit == bad).all()
    o[100:, 2:, 17] = want[0][100:, 2:, 17].to(BF16)
    ref.check_chunk(o, lse, want, BF16)


def test_pages_that_are_not_there():
    """Read as zeros and reported; other requests are whole."""
    c = Case([(20, 100), (30, 50)], 2, 1, F16, seed=10)
    want = c.reference()
    c.table[0, 2], c.table[0, 4] = -1, 10 ** 6
    o, lse = c.run()
    assert pkc.device_status(c.ws) == 4
    ref.check_chunk(o, lse, want, F16, slice(20, 50))
    assert torch.isfinite(o).all()
    k, v = c.k.clone(), c.v.clone()
    for t, j in ((c.table, 2), (c.table, 4)):
        spare = [p for p in range(k.shape[0]) if p not in c.table.tolist()[0] + c.table.tolist()[1]][j // 4]
        k[spare], v[spare] = 0, 0
        t[0, j] = spare
    ref.check_chunk(o, lse, ref.chunk(c.q, c.indptr, k, v, c.table, c.lens, c.scale), F16)


def test_a_table_that_is_too_narrow():
    c = Case([(9, 100), (8, 20)], 2, 1, F16, seed=11)
    want = c.reference()
    c.table = c.table[:, :4].contiguous()
    o, lse = c.run()
    assert pkc.device_status(c.ws) == 4
    ref.check_chunk(o, lse, want, F16, slice(9, 17))


def test_bad_ranges_and_lengths():
    c = Case([(5, 20), (6, 30), (7, 40)], 2, 1, F16, seed=12)
    want = c.reference()
    c.lens[1] = -4
    o, lse = c.run()
    assert pkc.device_status(c.ws) == 7
    ref.check_chunk(o, lse, want, F16, list(range(5)) + list(range(11, 18)))
    assert (o[5:11] == 7).all()
    c.lens[1] = 36
    c.indptr = [0, 5, 11, 40]
    o, lse = c.run()
    assert pkc.device_status(c.ws) == 7
    ref.check_chunk(o, lse, want, F16, slice(0, 11))
    c.indptr = [0, 5, 3, 18]
    c.run()
    assert pkc.device_status(c.ws) == 7
    c.indptr = [-2, 5, 11, 18]
    o, lse = c.run()
    assert pkc.device_status(c.ws) == 7
    ref.check_chunk(o, lse, want, F16, slice(5, 18))


def test_many_requests():
    rng = np.random.default_rng(13)
    reqs = [(int(rng.integers(0, 4)), int(rng.integers(0, 60))) for _ in range(700)]
    Case(reqs, 2, 1, BF16, seed=13).check()


def test_again_gives_the_same_bits():
    c = Case([(3, 5000), (200, 1000), (1, 2000)], 8, 1, BF16, seed=14)
    o, lse = c.check()
    for _ in range(3):
        p, l = c.run()
        assert torch.equal(o, p) and torch.equal(lse, l)


def test_empty_calls():
    c = Case([(0, 20), (0, 0)], 2, 1, F16, lead=3, seed=15)
    o, lse = c.run()
    assert (o == 7).all() and (lse == 7).all() and pkc.device_status(c.ws) == 0
    q = torch.empty((0, 2, 128), dtype=F16, device="cuda")
    o, lse = pkc.paged_chunk_state(q, torch.zeros(3, dtype=I32, device="cuda"), c.k.cuda(), c.v.cuda(), c.table.cuda(),
                                   torch.tensor(c.lens, dtype=I32, device="cuda"), c.scale, c.ws)
    assert o.shape == (0, 2, 128) and lse.shape == (0, 2)


def test_graph_other_stream_and_two_workspaces():
    a, b = Case([(3, 2000), (120, 60)], 8, 2, BF16, seed=16), Case([(50, 900), (1, 70)], 4, 2, F16, seed=17)
    want = [x.check() for x in (a, b)]
    keep = []
    for c in (a, b):
        keep.append((c.q.cuda(), torch.tensor(c.indptr, dtype=I32, device="cuda"), c.k.cuda(), c.v.cuda(), c.table.cuda(),
                     torch.tensor(c.lens, dtype=I32, device="cuda"), c.scale, c.ws))
    streams = [torch.cuda.Stream() for _ in keep]
    for _ in range(5):  # two at once
        got = []
        for s, args in zip(streams, keep):
            s.wait_stream(torch.cuda.current_stream())
            got.append(pkc.paged_chunk_state(*args, stream=s))
        torch.cuda.synchronize()
        for (o, l), (p, m) in zip(want, got):
            assert torch.equal(o, p) and torch.equal(l, m)
    out = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    graphs = []
    for args, (o, l) in zip(keep, out):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkc.paged_chunk_state(*args, o=o, lse=l)
        graphs.append(g)
    for _ in range(3):
        for o, l in out:
            o.fill_(0), l.fill_(0)
        for g in graphs:
            g.replay()
        for (o, l), (p, m) in zip(want, out):
            assert torch.equal(o, p) and torch.equal(l, m)
    # the lengths are read at replay: one token fewer of the first request
    keep[0][5][0] -= 1
    graphs[0].replay()
    a.lens[0] -= 1
    w = a.reference()
    ref.check_chunk(*out[0], w, BF16)


def test_one_workspace_with_a_decode_plan():
    """The partial states lie at the workspace's end: an uploaded plan stays."""
    c = Case([(4, 700), (2, 300)], 8, 2, BF16, seed=18)
    lens = np.array(c.lens, np.int32)
    plan = pkc.plan(lens, 16)
    size = pkc.workspace_size(2, 8, 16, 0)
    c.ws = workspace(size)
    pkc.plan_upload(plan, c.ws)
    c.check()
    q = c.q[[3, 5]].cuda()  # the last rows see every token
    o, lse = pkc.paged_decode_state(q, torch.nan_to_num(c.k, 0).cuda(), torch.nan_to_num(c.v, 0).cuda(), c.table.cuda(), torch.tensor(c.lens, dtype=I32, device="cuda"),
                                    c.scale, c.ws, plan_buf=plan)
    want = [x[[3, 5]] for x in c.reference()]
    ref.check_chunk(o, lse, want, BF16)
    assert pkc.device_status(c.ws) == 0


def test_refuses():
    c = Case([(5, 20)], 2, 1, F16)
    ip, lens = torch.tensor(c.indptr, dtype=I32, device="cuda"), torch.tensor(c.lens, dtype=I32, device="cuda")
    q, k, v, t = c.q.cuda(), c.k.cuda(), c.v.cuda(), c.table.cuda()
    with pytest.raises(TypeError, match="dtype"):
        pkc.paged_chunk_state(q.bfloat16(), ip, k, v, t, lens, 0.1, c.ws)
    with pytest.raises(ValueError, match="shape"):
        pkc.paged_chunk_state(q, ip[:1], k, v, t, lens, 0.1, c.ws)
    with pytest.raises(ValueError, match="contiguous"):
        pkc.paged_chunk_state(q.transpose(0, 1).contiguous().transpose(0, 1), ip, k, v, t, lens, 0.1, c.ws)
    with pytest.raises(TypeError, match="out_dtype"):
        pkc.paged_chunk_state(q, ip, k, v, t, lens, 0.1, c.ws, out_dtype=BF16)
    with pytest.raises(pkc.PkcError):
        pkc.paged_chunk_state(q, ip, k, v, t, lens, 0.1, c.ws[:-256])
    with pytest.raises(pkc.PkcError):
        pkc.paged_chunk_state(q, ip, k, v, t, lens, -0.1, c.ws)
    with pytest.raises(pkc.PkcError):
        pkc.paged_chunk_state(q, ip, k, v, t, lens, 0.1, c.ws, window=-1)


@pytest.mark.parametrize("below", [12.0, 20.0, 25.5, 28.0])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_many_small_weights_beside_a_large_one(dtype, below):
    """The first token holds the attention, 1500 others lie so many powers of two below it, and only they have a value.

    Each weight is half a step of its type off, and in fp16, where the largest stands for 2^6 or more and the smallest
    step is 2^-24, at most 2^-31 of the largest.  The scores are float32 products of one term: 2^-22 of the exponent,
    and as much again for the exponential; the sum and the quotient 2^-19.  LSE, up to 29 in powers of two: 2^-23 of
    it for the scale times log2(e), and half a step each, 2^-20, for the sum with the logarithm, the factor and the
    product."""
    c = Case([(1, 1500)], 1, 1, dtype, seed=21, scale=1.0)
    c.q[:] = 0
    c.q[..., 0] = 1.0
    key = torch.tensor(below * math.log(2)).to(dtype)
    for x, first, other in ((c.k, key, 0.0), (c.v, 0.0, 1.0)):
        page, rest = int(c.table[0, 0]), ~x.isnan()
        x[rest] = other
        x[page, 0, 0, :] = first
    c.k[..., 1:] = 0
    o, lse = c.run(out_dtype=torch.float32)
    assert pkc.device_status(c.ws) == 0
    w = math.exp(-float(key))
    want = 1500 * w / (1 + 1500 * w)
    tol = (ref.HALF_STEP[dtype] + 2.0 ** -17) * want + (1500 * 2.0 ** -31 if dtype == F16 else 0)
    assert float((o.double().cpu() - want).abs().max()) <= tol
    assert float((lse.double().cpu() - math.log(math.exp(float(key)) + 1500)).abs().max()) <= 2.0 ** -17


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1)])
def test_a_query_that_is_not_a_number(hq, hkv):
    """Its states are NaN, LSE too, whether its item is cut or not; the other rows are whole."""
    for reqs in ([(3, 6000)], [(3, 600)]):
        c = Case(reqs, hq, hkv, BF16, seed=22)
        want = c.reference()
        c.q[1, :, 7] = math.nan
        o, lse = c.run()
        assert pkc.device_status(c.ws) == 0
        assert o[1].isnan().all() and lse[1].isnan().all()
        ref.check_chunk(o, lse, want, BF16, [0, 2])


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_scores_that_rise_from_tile_to_tile(dtype):
    """Each tile of 128 keys lies 2^23 to 2^29 above the one before: what is formed against the old reference is
    infinite in fp16 and formed again."""
    c = Case([(150, 700), (1, 1000), (260, 0)], 4, 1, dtype, seed=23, scale=1.0)
    c.q *= 0.1
    c.q[..., 0] = 1.0
    for b, n in enumerate(c.lens):
        for t in range(n):
            c.k[c.table[b, t // 16], t % 16, :, 0] = 16.0 * (t // 128) + 4.0 * (t // 128 % 2)
    c.check()


@pytest.mark.parametrize("hq,hkv", [(3, 3), (5, 5), (12, 3), (7, 7), (40, 5)])
def test_odd_numbers_of_heads(hq, hkv):
    Case([(37, 91), (1, 300), (3, 0)], hq, hkv, F16, seed=hq).check()


def shifted(x, by):
    """x in memory that begins `by` bytes behind a multiple of 256."""
    n, size = x.numel(), x.element_size()
    buf = torch.zeros(n + 256 // size, dtype=x.dtype, device="cuda")
    out = buf[by // size:by // size + n].view(x.shape)
    out.copy_(x)
    assert out.data_ptr() % 256 == by
    return out


@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_least_alignment(out_dtype):
    """Rows, pools and results on 16 bytes, whole numbers and LSE on 4."""
    c = Case([(37, 91), (1, 1900), (140, 0)], 4, 2, F16, seed=24)
    o = shifted(torch.full(c.q.shape, 7.0, dtype=out_dtype or F16), 16)
    lse = shifted(torch.full(c.q.shape[:2], 7.0), 4)
    pkc.paged_chunk_state(shifted(c.q, 48), shifted(torch.tensor(c.indptr, dtype=I32), 4), shifted(c.k, 16), shifted(c.v, 80), shifted(c.table, 4),
                          shifted(torch.tensor(c.lens, dtype=I32), 12), c.scale, c.ws, o=o, lse=lse)
    ref.check_chunk(o, lse, c.reference(), o.dtype)
    assert pkc.device_status(c.ws) == 0
