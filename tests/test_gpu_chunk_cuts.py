"""Chunk attention where items are cut over several blocks: pieces in several words of the ready
bits, both halves, windows, rows computed again in a piece; against the definition in 64 bits."""
import math

import pytest
import torch

import paged_kv_cascade_gb300 as pkc
import prompt_reference as ref
from chunk_cuts import CASES, pieces
from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def is_cut(reqs, hq, hkv, causal=True, window=0):
    blocks = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    return any(len(of) > 1 for _, _, of in pieces(reqs, hkv, hq // hkv, blocks, causal, window))


@pytest.mark.parametrize("name", list(CASES))
def test_cut_items(name):
    reqs, hq, hkv, causal, window = CASES[name]
    assert is_cut(reqs, hq, hkv, causal, window)
    c = Case(reqs, hq, hkv, BF16 if len(name) % 2 else F16, seed=31, lead=7, trail=5)
    o, lse = c.check(causal, window)
    for _ in range(3):  # bits left behind would show
        p, l = c.run(causal, window)
        assert torch.equal(o, p) and torch.equal(lse, l)
    o32, lse32 = c.run(causal, window, out_dtype=torch.float32)
    assert torch.equal(lse, lse32) and torch.equal(o, o32.to(o.dtype))
    assert pkc.device_status(c.ws) == 0


def test_cut_items_of_all_sizes_in_turn():
    """One workspace, calls whose pieces share words of the ready bits in other ways each time."""
    cases = [Case(*CASES[name][:3], BF16, seed=32) for name in ("several items", "beside others", "both halves", "five words")]
    ws = cases[0].ws
    first = []
    for c in cases:
        c.ws = ws
        first.append(c.run())
    for i in (3, 1, 0, 2, 1, 3):
        o, lse = cases[i].run()
        assert torch.equal(o, first[i][0]) and torch.equal(lse, first[i][1])
    assert pkc.device_status(ws) == 0
    ref.check_chunk(*first[1], cases[1].reference(), BF16)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("hq,hkv,dtype", [(4, 1, F16), (1, 1, BF16)])
def test_values_that_are_not_finite_in_a_cut_item(hq, hkv, dtype, bad):
    """Rows of a piece computed again: a value before a window's begin and one among the new tokens reach the rows
    that attend to them and no others."""
    reqs = [(20, 5000), (3, 4000)]
    c = Case(reqs, hq, hkv, dtype, seed=33)
    assert is_cut(reqs, hq, hkv) and is_cut(reqs, hq, hkv, True, 2000)
    want, want_window = c.reference(), c.reference(window=2000)
    for t, dim in ((5010, 5), (3006, 40)):
        c.v[c.table[0, t // 16], t % 16, 0, dim] = bad
    # row i stands at 5000 + i; a window of 2000 begins at 3001 + i
    o, lse = c.run(window=2000)
    assert pkc.device_status(c.ws) == 0
    ref.check_chunk(o, lse, want_window, dtype, [6, 7, 8, 9, 20, 21, 22])
    got = o.cpu()
    assert not torch.isfinite(got[:6, :, 40]).any() and not torch.isfinite(got[10:20, :, 5]).any()
    got[:6, :, 40] = want_window[0][:6, :, 40].to(dtype)
    got[10:20, :, 5] = want_window[0][10:20, :, 5].to(dtype)
    ref.check_chunk(got, lse, want_window, dtype)
    o, lse = c.run()  # all rows attend to token 3006
    got = o.cpu()
    assert not torch.isfinite(got[:20, :, 40]).any() and not torch.isfinite(got[10:20, :, 5]).any()
    got[:20, :, 40] = want[0][:20, :, 40].to(dtype)
    got[10:20, :, 5] = want[0][10:20, :, 5].to(dtype)
    ref.check_chunk(got, lse, want, dtype)


@pytest.mark.parametrize("dtype,q_exp,k_exp", [(F16, 14, 8), (BF16, 30, 40)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_far_out_in_a_cut_item(dtype, q_exp, k_exp, sign):
    """As for the items that are not cut: a score is its key's dim 0 times a power of two, two different ones lie more than
    2^9 apart, so the largest one's values come out; each is off by two half steps and 2^-19 of a few roundings, and a
    merge of equal maxima by as much as a sum's."""
    reqs = [(30, 3000), (2, 2500)]
    c = Case(reqs, 4, 1, dtype, seed=34, scale=1.0)
    assert is_cut(reqs, 4, 1)
    gen = torch.Generator().manual_seed(35)
    c.q[:] = 0
    c.q[..., 0] = 2.0 ** q_exp
    rank = torch.randint(1, 100, c.k.shape[:3], generator=gen)
    c.k[..., 0] = torch.where(c.k[..., 0].isnan(), c.k[..., 0], (sign * rank * 2.0 ** k_exp).to(dtype))
    o, lse = c.run()
    assert pkc.device_status(c.ws) == 0
    want, want_lse, _, _ = c.reference()
    assert float(((o.double().cpu() - want).abs() - 2 * ref.HALF_STEP[dtype] * want.abs()).max()) <= 2.0 ** -19
    assert torch.all((lse.double().cpu() - want_lse).abs() <= 2.0 ** -21 * want_lse.abs())


def test_pages_that_are_not_there_in_a_cut_item():
    """Zeros in one piece, reported; the other request is whole."""
    reqs = [(5, 6000), (3, 5000)]
    c = Case(reqs, 4, 1, F16, seed=36)
    assert is_cut(reqs, 4, 1)
    want = c.reference()
    for j in (100, 101, 300):
        c.table[0, j] = -1 if j % 2 else 10 ** 6
    o, lse = c.run()
    assert pkc.device_status(c.ws) == 4
    ref.check_chunk(o, lse, want, F16, slice(5, 8))
    assert torch.isfinite(o).all()
    spare = [p for p in range(c.k.shape[0]) if p not in c.table.flatten().tolist()]
    c.k[spare], c.v[spare] = 0, 0
    for i, j in enumerate((100, 101, 300)):
        c.table[0, j] = spare[i]
    ref.check_chunk(o, lse, c.reference(), F16)


@pytest.mark.parametrize("dtype,score", [(F16, 6.875), (BF16, 8.875)])
@pytest.mark.parametrize("late", [130, 1000, 1530])
def test_a_late_key_that_holds_the_row(dtype, score, late):
    """Single tokens whose attention is on one key, less than 2^13 above the first tile's best: its weight is the row's
    largest, so it is exact, and the others' half steps are all that is lost.

    The scores are products of one term: 2^-17 of a weight for them and the exponential.  An error e of a weight w moves
    O by w e |v - O|; in fp16 e w is at least 2^-31 of the largest.  O is summed in 32 bits, 16 keys at a time: at most
    a step of 2^-23 of its size for each of n / 16 additions, which need not round to nearest, and for eight roundings
    of the sum, the quotient and the merge of pieces."""
    reqs = [(1, 1530), (1, 5000)]
    c = Case(reqs, 4, 1, dtype, seed=37, scale=1.0)
    c.q[:] = 0
    c.q[..., 0] = 1.0
    c.k[..., 0] = torch.where(c.k[..., 0].isnan(), c.k[..., 0], torch.full_like(c.k[..., 0], -8.0))
    for b in range(2):
        for t, x in ((3, 0.0), (late, score)):
            c.k[c.table[b, t // 16], t % 16, 0, 0] = x
    o, lse = c.run(out_dtype=torch.float32)
    assert pkc.device_status(c.ws) == 0
    for b, n in enumerate(c.lens):
        pages = c.table[b, :-(-n // 16)].long()
        x, v = c.k[pages, :, 0, 0].flatten()[:n].double(), c.v[pages, :, 0].flatten(0, 1)[:n].double()
        w = torch.softmax(x, 0)
        want = w @ v
        w[late] = 0
        tol = (ref.HALF_STEP[dtype] + 2.0 ** -17) * (w @ (v - want).abs()) + 2.0 ** -17 * (v[late] - want).abs() + (n / 16 + 8) * 2.0 ** -23 * (want.abs() + w @ v.abs())
        if dtype == F16:
            tol += 2.0 ** -31 * (v - want).abs().sum(0)
        assert float(((o[b].double().cpu() - want).abs() - tol).max()) <= 0
        assert torch.all((lse[b].double().cpu() - torch.logsumexp(x, 0)).abs() <= 2.0 ** -18)
