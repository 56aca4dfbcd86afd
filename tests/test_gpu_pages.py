"""Pages and slots for new tokens, and pages given back, against the plain definitions."""
import numpy as np
import pytest
import torch

import paged_kv_cascade_gb300 as pkc
import prompt_reference as ref

pytestmark = pytest.mark.gpu
I32 = torch.int32


def workspace(n=256):
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    pkc.workspace_init(ws)
    return ws


def state(batch, page, num_pages, most, stride, seed, held=0):
    """Random lengths whose pages come from a permuted pool; `held` further entries behind each length."""
    rng = np.random.default_rng(seed)
    perm = rng.permutation(num_pages).tolist()
    lens, table = [], []
    for _ in range(batch):
        n = int(rng.integers(0, min(most, (stride - held) * page) + 1))
        need = -(-n // page) + held
        if need > len(perm):
            n, need = 0, 0
        row = [perm.pop() for _ in range(need)]
        lens.append(n)
        table.append(row + [-1] * (stride - len(row)))
    return lens, table, set(perm)


class Run:
    def __init__(self, lens, table, free, page, num_pages):
        self.lens, self.table, self.free, self.page, self.num_pages = lens, [list(r) for r in table], set(free), page, num_pages
        self.d_lens = torch.tensor(lens, dtype=I32, device="cuda")
        self.d_table = torch.tensor(table, dtype=I32, device="cuda")
        self.d_free = ref.pool_words(free, num_pages).cuda()
        self.ws = workspace()

    def release(self, want=0):
        pkc.release_pages(self.d_table, self.d_lens, self.d_free, self.page, self.num_pages, self.ws)
        ref.release(self.table, self.lens, self.free, self.page)
        self.check(want)

    def assign(self, new, lead=0, trail=0, want=None, in_place=False):
        indptr = [lead]
        for n in new:
            indptr.append(indptr[-1] + n)
        total = indptr[-1] + trail
        out = self.d_lens if in_place else None
        got = pkc.assign_pages(self.d_table, self.d_lens, torch.tensor(indptr, dtype=I32, device="cuda"), total, self.d_free,
                               self.page, self.num_pages, self.ws, seqlens_out=out)
        slots, pos, lens, status = ref.assign(self.table, self.lens, indptr, total, self.free, self.page)
        assert got[0].tolist() == slots
        assert got[1].tolist() == pos
        assert got[2].tolist() == lens
        self.check(status if want is None else want)
        if in_place:
            self.lens = lens
        return got

    def check(self, want):
        assert self.d_table.tolist() == self.table
        assert ref.pool_set(self.d_free, self.num_pages) == self.free
        assert pkc.device_status(self.ws) == want


@pytest.mark.parametrize("batch,page,num_pages,most_new", [
    (1, 16, 1, 16), (1, 1, 33, 33), (3, 16, 40, 5), (5, 7, 300, 60), (64, 16, 8000, 1), (130, 20, 4096, 90),
    (1500, 16, 70001, 40), (7, 64, 5000, 9000), (40, 8, 200000, 3000),
])
def test_assign(batch, page, num_pages, most_new):
    rng = np.random.default_rng(batch + page)
    stride = max(1, num_pages // batch)
    lens, table, free = state(batch, page, num_pages, stride * page // 2, stride, 5)
    run = Run(lens, table, free, page, num_pages)
    run.assign(rng.integers(0, most_new + 1, batch).tolist())


def test_steps_until_the_pool_is_empty():
    """One token each, lengths grown in place, until requests find no pages;
    then a request ends and others go on with its pages."""
    page, num_pages = 4, 37
    lens, table, free = state(9, page, num_pages, 10, 40, 3)
    run = Run(lens, table, free, page, num_pages)
    for _ in range(12):
        run.assign([1] * 9, in_place=True)
    assert not run.free
    run.lens[2] = 0
    run.d_lens[2] = 0
    run.release()
    assert run.free
    run.assign([1] * 9, lead=2, trail=3, in_place=True)


def test_release_gives_back_in_any_order():
    lens, table, free = state(60, 16, 5000, 900, 70, 9, held=5)
    run = Run(lens, table, free, 16, 5000)
    before = set(run.free)
    run.release()
    assert len(run.free) > len(before)
    run.assign([17] * 60)
    run.release()  # the lengths did not grow: the same pages come back
    run.assign([17] * 60)


def test_rows_of_no_request_and_empty_batches():
    run = Run([3, 0], [[1, -1], [-1, -1]], {0, 2}, 4, 3)
    slots, pos, _ = run.assign([0, 2], lead=4, trail=2)
    assert slots.tolist() == [-1] * 4 + [0, 1] + [-1] * 2 and pos.tolist() == [0] * 4 + [0, 1] + [0] * 2
    run.assign([0, 0])
    s, p, n = pkc.assign_pages(run.d_table[:0], run.d_lens[:0], torch.zeros(1, dtype=I32, device="cuda"), 3, run.d_free, 4, 3, run.ws)
    assert s.tolist() == [-1] * 3 and p.tolist() == [0] * 3 and n.numel() == 0
    pkc.release_pages(run.d_table[:0], run.d_lens[:0], run.d_free, 4, 3, run.ws)
    run.check(0)


@pytest.mark.parametrize("num_pages", [700, 1400])
def test_many_tokens(num_pages):
    """More tokens than one launch places, with and without enough pages, rows of no request on both sides."""
    rng = np.random.default_rng(7)
    new = rng.integers(0, 900, 25).tolist()
    new[3] = new[24] = 0
    lens, table, free = state(25, 16, num_pages, 200, 80, 11)
    run = Run(lens, table, free, 16, num_pages)
    run.assign(new, lead=37, trail=401, in_place=True)
    run.assign(new)


def test_many_tokens_of_nobody():
    run = Run([3, 0], [[1, -1], [-1, -1]], {0, 2}, 4, 3)
    table, lens = run.d_table[:0], run.d_lens[:0]
    s, p, _ = pkc.assign_pages(table, lens, torch.zeros(1, dtype=I32, device="cuda"), 9000, run.d_free, 4, 3, run.ws)
    assert (s == -1).all() and (p == 0).all()
    wrong = torch.tensor([0, 8999, 8000], dtype=I32, device="cuda")
    s, p, n = pkc.assign_pages(run.d_table, run.d_lens, wrong, 9000, run.d_free, 4, 3, run.ws)
    assert (s == -1).all() and n.tolist() == [3, 0]
    run.check(7)


def test_served_in_order():
    """The second request is too large for what is left; a third that needs no page is served, a fourth that does is not."""
    run = Run([0, 0, 1, 0], [[-1] * 4, [-1] * 4, [9, -1, -1, -1], [-1] * 4], {3, 4, 5}, 4, 10)
    run.assign([5, 8, 2, 1])
    assert run.table[0][:2] == [3, 4] and run.free == {5}


def test_bits_behind_the_pool_are_kept():
    words = torch.full((1,), -1, dtype=I32, device="cuda")
    ws, table = workspace(), torch.full((1, 40), -1, dtype=I32, device="cuda")
    pkc.assign_pages(table, torch.zeros(1, dtype=I32, device="cuda"), torch.tensor([0, 11], dtype=I32, device="cuda"), 11, words, 1, 10, ws)
    assert pkc.device_status(ws) == 8 and words.tolist() == [-1]  # ten pages, eleven asked for
    pkc.assign_pages(table, torch.zeros(1, dtype=I32, device="cuda"), torch.tensor([0, 10], dtype=I32, device="cuda"), 10, words, 1, 10, ws)
    assert pkc.device_status(ws) == 0 and words.tolist() == [-1024] and table[0, :10].tolist() == list(range(10))


def test_what_cannot_be_served_is_left():
    """A negative length, a table that is too narrow, a partly filled page that is not there."""
    lens = torch.tensor([-1, 7, 5, 6, 2], dtype=I32, device="cuda")
    table = torch.tensor([[0, 1], [2, 3], [4, -1], [5, 99], [6, -1]], dtype=I32, device="cuda")
    free, ws = ref.pool_words({8, 9}, 12).cuda(), workspace()
    indptr = torch.tensor([0, 1, 3, 4, 5, 8], dtype=I32, device="cuda")
    slots, pos, out = pkc.assign_pages(table, lens, indptr, 8, free, 4, 12, ws)
    assert pkc.device_status(ws) == 4
    assert slots.tolist() == [-1, -1, -1, -1, -1, 26, 27, 32] and out.tolist() == [-1, 7, 5, 6, 5]
    assert pos.tolist() == [-1, 7, 8, 5, 6, 2, 3, 4]
    assert table.tolist() == [[0, 1], [2, 3], [4, -1], [5, 99], [6, 8]] and ref.pool_set(free, 12) == {9}


@pytest.mark.parametrize("indptr,total", [([0, 3, 2], 4), ([-1, 1, 2], 2), ([0, 2, 5], 4)])
def test_bad_ranges_serve_nobody(indptr, total):
    lens, table = torch.tensor([1, 2], dtype=I32, device="cuda"), torch.tensor([[0, -1], [1, -1]], dtype=I32, device="cuda")
    free, ws = ref.pool_words({2, 3}, 4).cuda(), workspace()
    slots, pos, out = pkc.assign_pages(table, lens, torch.tensor(indptr, dtype=I32, device="cuda"), total, free, 4, 4, ws)
    assert pkc.device_status(ws) == 7 and slots.tolist() == [-1] * total and out.tolist() == [1, 2]
    assert table.tolist() == [[0, -1], [1, -1]] and ref.pool_set(free, 4) == {2, 3}


def test_release_reports():
    """A page that is free already, one held twice, one outside the pool, a negative length."""
    table = torch.tensor([[0, 5, 5, 3], [1, 77, -1, 4], [6, 7, 8, 9]], dtype=I32, device="cuda")
    lens, ws = torch.tensor([4, 4, -2], dtype=I32, device="cuda"), workspace()
    free = ref.pool_words({3}, 12).cuda()
    pkc.release_pages(table, lens, free, 4, 12, ws)
    assert pkc.device_status(ws) in (4, 7)
    assert table.tolist() == [[0, -1, -1, -1], [1, 77, -1, -1], [6, 7, 8, 9]]
    assert ref.pool_set(free, 12) == {3, 4, 5}


def test_graph_and_another_stream():
    lens, table, free = state(20, 16, 3000, 300, 60, 4, held=2)
    run = Run(lens, table, free, 16, 3000)
    indptr = torch.arange(21, dtype=I32, device="cuda") * 33
    args = (run.d_table, run.d_lens, indptr, 660, run.d_free, 16, 3000, run.ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkc.release_pages(run.d_table, run.d_lens, run.d_free, 16, 3000, run.ws, stream=side)
    slots, pos, out = (torch.empty(660, dtype=torch.int64, device="cuda"), torch.empty(660, dtype=I32, device="cuda"), torch.empty(20, dtype=I32, device="cuda"))
    side.wait_stream(torch.cuda.current_stream())
    pkc.assign_pages(*args, slots=slots, positions=pos, seqlens_out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = slots.clone(), pos.clone(), out.clone(), run.d_table.clone(), run.d_free.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkc.release_pages(run.d_table, run.d_lens, run.d_free, 16, 3000, run.ws)
        pkc.assign_pages(*args, slots=slots, positions=pos, seqlens_out=out)
    for _ in range(3):
        slots.fill_(-7)
        g.replay()
    for a, b in zip((slots, pos, out, run.d_table, run.d_free), want):
        assert torch.equal(a, b)
    ref.release(run.table, lens, run.free, 16)
    ref.assign(run.table, lens, indptr.tolist(), 660, run.free, 16)
    run.check(0)


@pytest.mark.parametrize("batch,most_new", [(50, 1500), (16384, 3)])
@pytest.mark.parametrize("num_pages", [40_001, 2 ** 21, 2 ** 21 + 1, 2 ** 26])
def test_free_pages_far_apart(num_pages, batch, most_new):
    """Few free pages, some side by side, in pools up to the largest; the largest batch."""
    rng = np.random.default_rng(num_pages % 1000 + batch)
    free = set(rng.integers(0, num_pages, 6000).tolist()) | {0, num_pages - 1} | set(range(9000, 9700))
    page, new = 16, rng.integers(0, most_new + 1, batch).tolist()
    stride = 4 + -(-most_new // page)
    lens, table, held = [], [], num_pages // 2
    for _ in range(batch):
        n = int(rng.integers(0, 4 * page))
        row = []
        while len(row) < -(-n // page):  # any pages that are not free
            held = (held + 1) % num_pages
            if held not in free:
                row.append(held)
        lens.append(n)
        table.append(row + [-1] * (stride - len(row)))
    indptr = np.concatenate(([0], np.cumsum(new))).tolist()
    d_table, d_lens, d_free = torch.tensor(table, dtype=I32, device="cuda"), torch.tensor(lens, dtype=I32, device="cuda"), ref.pool_words(free, num_pages).cuda()
    ws = workspace()
    for _ in range(2):
        got = pkc.assign_pages(d_table, d_lens, torch.tensor(indptr, dtype=I32, device="cuda"), indptr[-1], d_free, page, num_pages, ws, seqlens_out=d_lens)
        slots, pos, lens, status = ref.assign(table, lens, indptr, indptr[-1], free, page)
        assert got[0].tolist() == slots and got[1].tolist() == pos and got[2].tolist() == lens
        assert d_table.tolist() == table and torch.equal(d_free.cpu(), ref.pool_words(free, num_pages))
        assert pkc.device_status(ws) == status
        pkc.workspace_init(ws)
    d_lens.zero_()
    pkc.release_pages(d_table, d_lens, d_free, page, num_pages, ws)
    ref.release(table, [0] * batch, free, page)
    want = ref.pool_words(free, num_pages)
    assert torch.equal(d_free.cpu(), want) and (d_table == -1).all()


@pytest.mark.parametrize("total", [3, 8192, 9000])
def test_no_requests_need_no_arrays(total):
    """A batch of none: its arrays may be NULL, and every token is nobody's."""
    slots, pos = torch.full((total,), 7, dtype=torch.int64, device="cuda"), torch.full((total,), 7, dtype=I32, device="cuda")
    ws = workspace()
    stream = torch.cuda.current_stream().cuda_stream
    assert pkc.lib().pkc_assign_pages(None, 4, None, None, total, 0, 16, 1000, None, slots.data_ptr(), pos.data_ptr(), None, ws.data_ptr(),
                                      ws.numel(), stream) == 0
    assert (slots == -1).all() and (pos == 0).all() and pkc.device_status(ws) == 0


def test_many_tokens_captured_and_on_another_stream():
    """Both launches of a call for many tokens in a graph, replayed over a table and a pool that are put back."""
    rng = np.random.default_rng(8)
    new = rng.integers(0, 900, 25).tolist()
    lens, table, free = state(25, 16, 1400, 200, 80, 12)
    run = Run(lens, table, free, 16, 1400)
    indptr = [5] + (5 + np.cumsum(new)).tolist()
    total = indptr[-1] + 11
    d_indptr = torch.tensor(indptr, dtype=I32, device="cuda")
    assert total > 8192
    slots, pos, out = (torch.empty(total, dtype=torch.int64, device="cuda"), torch.empty(total, dtype=I32, device="cuda"), torch.empty(25, dtype=I32, device="cuda"))
    old = run.d_table.clone(), run.d_free.clone()

    def call(stream=None):
        pkc.assign_pages(run.d_table, run.d_lens, d_indptr, total, run.d_free, 16, 1400, run.ws, slots=slots, positions=pos, seqlens_out=out, stream=stream)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    want = ref.assign(run.table, run.lens, indptr, total, run.free, 16)
    side = torch.cuda.Stream()
    for replay in (True, True, False, True):
        run.d_table.copy_(old[0])
        run.d_free.copy_(old[1])
        for x in (slots, pos, out):
            x.fill_(-9)
        if replay:
            g.replay()
        else:
            side.wait_stream(torch.cuda.current_stream())
            call(side)
            torch.cuda.current_stream().wait_stream(side)
        assert slots.tolist() == want[0] and pos.tolist() == want[1] and out.tolist() == want[2]
        run.check(want[3])
