"""A prompt's way into the cache, without a GPU: the entry points' refusals,
the frequencies, the pool's map, and the plain definitions on worked examples."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cascade_gb300 as pkc
import prompt_reference as ref
from paged_kv_cascade_gb300 import build as pkc_build

F, WS, OUT = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x100000), ctypes.c_void_p(0x80000)
OFF8, OFF4, OFF2 = ctypes.c_void_p(0x1008), ctypes.c_void_p(0x1004), ctypes.c_void_p(0x1002)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    pkc_build.build()
    return pkc.lib()


def variants(good, changes):
    """(position, value, expected code) applied one at a time to the good arguments."""
    for pos, val, code in changes:
        yield good[:pos] + [val] + good[pos + 1:], code


def test_release_refuses(L):
    # table stride lens batch ps pages free ws bytes stream
    good = [F, 4, F, 2, 16, 10, F, WS, 1 << 20, None]
    for args, code in variants(good, [
            (0, None, 1), (2, None, 1), (6, None, 1), (0, OFF2, 1), (2, OFF2, 1), (6, OFF2, 1), (1, 0, 1), (3, -1, 1),
            (3, 16385, 2), (4, 0, 1), (4, 2 ** 30, 2), (5, -1, 1), (5, 2 ** 26 + 1, 2), (7, None, 3), (7, OFF4, 3),
            (8, 255, 3)]):
        assert L.pkc_release_pages(*args) == code, (args, L.pkc_last_error())
    assert L.pkc_release_pages(*good[:3], 0, *good[4:]) == 0


def test_assign_refuses(L):
    # table stride lens indptr total batch ps pages free slots positions out ws bytes stream
    good = [F, 4, F, F, 5, 2, 16, 10, F, F, F, F, WS, 1 << 20, None]
    for args, code in variants(good, [
            (0, None, 1), (2, None, 1), (3, None, 1), (8, None, 1), (9, None, 1), (10, None, 1), (0, OFF2, 1), (3, OFF2, 1),
            (8, OFF2, 1), (9, OFF4, 1), (10, OFF2, 1), (11, OFF2, 1), (1, 0, 1), (4, -1, 1), (5, -1, 1), (5, 16385, 2),
            (6, 0, 1), (6, 2 ** 30, 2), (7, -1, 1), (7, 2 ** 26 + 1, 2), (12, None, 3), (13, 255, 3)]):
        assert L.pkc_assign_pages(*args) == code, (args, L.pkc_last_error())
    assert L.pkc_assign_pages(*good[:4], 0, 0, *good[6:]) == 0


def test_rope_refuses(L):
    # q qs k v kvs pos slots freq rd inter amp total hq hkv d qo kc vc ps pages ksc vsc dtype kvdtype ws bytes stream
    good = [F, 1024, F, F, 256, F, F, F, 128, 0, 1.0, 5, 8, 2, 128, F, F, F, 16, 10, 1.0, 1.0, 1, 1, WS, 1 << 20, None]
    for args, code in variants(good, [
            (0, None, 1), (2, None, 1), (3, None, 1), (5, None, 1), (6, None, 1), (7, None, 1), (15, None, 1),
            (16, None, 1), (17, None, 1), (0, OFF8, 1), (2, OFF8, 1), (3, OFF8, 1), (15, OFF8, 1), (16, OFF8, 1),
            (17, OFF8, 1), (6, OFF4, 1), (7, OFF4, 1), (5, OFF2, 1), (1, 1016, 1), (1, 1028, 1), (1, 0, 1), (4, 248, 1),
            (4, -256, 1), (8, 0, 1), (8, 130, 1), (8, 7, 1), (8, 24, 2), (9, 2, 1), (10, NAN, 1), (10, INF, 1),
            (11, -1, 1), (12, 0, 1), (13, 0, 1), (12, 2 ** 16 + 1, 2), (14, 64, 2), (18, 0, 1), (19, -1, 1),
            (19, 2 ** 31, 2), (20, 2.0, 1), (20, 0.0, 1), (21, NAN, 1), (22, 0, 1), (22, 3, 1), (23, 2, 1), (23, 4, 1),
            (24, None, 3), (25, 100, 3)]):
        assert L.pkc_rope_append_kv(*args) == code, (args, L.pkc_last_error())
    fp8 = good[:23] + [3] + good[24:]
    for args, code in variants(fp8, [(20, 0.0, 1), (20, -1.0, 1), (21, INF, 1), (21, NAN, 1), (20, 1e-40, 1)]):
        assert L.pkc_rope_append_kv(*args) == code
    assert L.pkc_rope_append_kv(*good[:11], 0, *good[12:]) == 0


def test_rope_refuses_outputs_on_its_inputs(L):
    """5 tokens of 8 query heads (2 KB) and 2 KV heads (512 bytes), parts of one projection of 13 heads (3328
    bytes) at 0x100000, or dense: q_out on q's rows, on q itself where they lie apart, on keys or values, by one element's worth."""
    base = 0x100000
    end = base + 4 * 3328  # the last token's row
    apart = [(base, 1664, base + 2048, base + 2560, 1664)]
    for q, qs, k, v, kvs in apart:
        for out in (base, base + 16, base - 16, base + 3328, end + 2048 - 16, base - 5 * 2048 + 16,  # q
                    base + 2048, base + 2560 + 512 - 16, end + 2048, end + 2560 + 512 - 16):  # k, v
            args = [q, qs, k, v, kvs, 0x1000, 0x1000, 0x1000, 128, 0, 1.0, 5, 8, 2, 128, out, 0x800000, 0x900000, 16, 10, 1.0, 1.0, 1, 1,
                    WS, 1 << 20, None]
            args = [ctypes.c_void_p(a) if i in (0, 2, 3, 5, 6, 7, 15, 16, 17) else a for i, a in enumerate(args)]
            assert L.pkc_rope_append_kv(*args) == 1 and b"overlap" in L.pkc_last_error(), hex(out)
    for out in (base + 16, base - 16, base + 0x8000, base + 0x8000 - 5 * 2048 + 16, base + 0x8000 + 5 * 512 - 16, base + 0x10000 + 16):  # dense
        args = [base, 1024, base + 0x8000, base + 0x10000, 256, 0x1000, 0x1000, 0x1000, 128, 0, 1.0, 5, 8, 2, 128, out, 0x800000, 0x900000, 16,
                10, 1.0, 1.0, 1, 1, WS, 1 << 20, None]
        args = [ctypes.c_void_p(a) if i in (0, 2, 3, 5, 6, 7, 15, 16, 17) else a for i, a in enumerate(args)]
        assert L.pkc_rope_append_kv(*args) == 1 and b"overlap" in L.pkc_last_error(), hex(out)


def test_chunk_refuses(L):
    need = pkc.chunk_workspace_size()
    assert need % 256 == 0 and L.pkc_chunk_workspace_size(None) == 1
    # q qip total kc vc table stride lens batch hq hkv d ps pages scale causal window ws bytes o lse dtype odt stream
    good = [F, F, 5, F, F, F, 4, F, 2, 16, 8, 128, 16, 10, 1.0, 1, 0, WS, need, OUT, F, 1, 1, None]
    for args, code in variants(good, [
            (0, None, 1), (1, None, 1), (3, None, 1), (4, None, 1), (5, None, 1), (7, None, 1), (19, None, 1),
            (20, None, 1), (0, OFF8, 1), (3, OFF8, 1), (4, OFF8, 1), (19, OFF8, 1), (20, OFF2, 1), (1, OFF2, 1),
            (2, -1, 1), (6, 0, 1), (8, -1, 1), (9, 12, 1), (9, 24, 2), (10, 0, 1), (11, 64, 2), (12, 0, 1),
            (12, 2 ** 30, 2), (13, -1, 1), (13, 2 ** 31, 2), (14, -1.0, 1), (14, NAN, 1), (14, INF, 1), (14, 3e38, 1),
            (15, 2, 1), (16, -1, 1), (17, None, 3), (17, OFF8, 3), (18, need - 1, 3), (21, 0, 1), (21, 3, 1), (22, 2, 1),
            (22, 3, 1)]):
        assert L.pkc_paged_chunk_state(*args) == code, (args, L.pkc_last_error())
    # o on q, on its last row, and as float32 with its own last row on q (5 rows of 16 heads)
    for o, q, out in ((0x1000, 0x1000, 1), (0x1000 + 79 * 256, 0x1000, 1), (0x1000, 0x1000 + 79 * 512, 0)):
        args = [ctypes.c_void_p(q)] + good[1:19] + [ctypes.c_void_p(o)] + good[20:22] + [out, None]
        assert L.pkc_paged_chunk_state(*args) == 1 and b"overlap" in L.pkc_last_error()
    assert L.pkc_paged_chunk_state(*good[:2], 0, *good[3:]) == 0
    assert L.pkc_paged_chunk_state(*good[:8], 0, *good[9:]) == 0


def test_binding_refuses_host_tensors():
    i32 = torch.int32
    bt, lens, ip = torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    ws, free = torch.zeros(256, dtype=torch.uint8), pkc.page_pool(10, "cpu")
    k, q = torch.zeros(4, 16, 2, 128).half(), torch.zeros(2, 4, 128).half()
    with pytest.raises(ValueError, match="CUDA"):
        pkc.release_pages(bt, lens, free, 16, 10, ws)
    with pytest.raises(ValueError, match="CUDA"):
        pkc.assign_pages(bt, lens, ip, 2, free, 16, 10, ws)
    with pytest.raises(TypeError, match="dtype"):
        pkc.assign_pages(bt.long(), lens, ip, 2, free, 16, 10, ws)
    with pytest.raises(ValueError, match="CUDA"):
        pkc.rope_append_kv(q, k[0, :2], k[0, :2], lens, lens.long(), torch.zeros(64).double(), k, k, ws)
    with pytest.raises(ValueError, match="CUDA"):
        pkc.paged_chunk_state(q, ip, k, k, bt, lens, 0.1, ws)
    with pytest.raises(TypeError, match="dtype"):
        pkc.paged_chunk_state(q.float(), ip, k.float(), k.float(), bt, lens, 0.1, ws)


def test_integers_that_a_c_int_would_cut():
    for bad in (2 ** 31, 2 ** 32 + 16, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="window must fit in 32 bits"):
            pkc._c_int("window", bad)
    assert pkc._c_int("window", 2 ** 31 - 1) == 2 ** 31 - 1


def test_frequencies():
    f, a = pkc.rope_frequencies(64, base=500.0, device="cpu")
    assert f.dtype == torch.float64 and a == 1.0
    assert all(abs(float(f[i]) - 500.0 ** (-2 * i / 64)) < 1e-15 for i in range(32))
    g, a = pkc.rope_frequencies(64, base=500.0, factor=4.0, device="cpu")
    assert a == 1.0 and torch.allclose(g, f / 4, rtol=1e-15, atol=0)
    g, a = pkc.rope_frequencies(64, base=500.0, factor=4.0, context=1024, device="cpu")
    assert a == pytest.approx(0.1 * math.log(4.0) + 1.0, abs=1e-15)
    for i in range(32):
        turns = 1024 * float(f[i]) / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 31))
        assert float(g[i]) == pytest.approx(float(f[i]) * (keep + (1 - keep) / 4), rel=1e-14)
    assert float(g[0]) == 1.0 and float(g[-1]) == pytest.approx(float(f[-1]) / 4, rel=1e-14)
    for bad in (dict(rotary_dim=0), dict(rotary_dim=7), dict(base=0.0), dict(factor=0.5), dict(factor=2.0, context=0),
                dict(factor=2.0, context=10, slow=3, fast=3)):
        with pytest.raises(ValueError):
            pkc.rope_frequencies(**{"device": "cpu", **bad})


@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 100])
def test_pool_map(n):
    w = pkc.page_pool(n, "cpu")
    assert w.dtype == torch.int32 and ref.pool_set(w, n) == set(range(n))
    assert torch.equal(w, ref.pool_words(range(n), n))
    with pytest.raises(ValueError):
        pkc.page_pool(-1, "cpu")


def test_assign_by_hand():
    """Page size 4, free pages 2 5 6 9: request 0 fills its page, request 1
    starts, request 2 crosses a page, request 3 finds too few left."""
    table = [[7, -1, -1], [-1, -1, -1], [3, -1, -1], [8, -1, -1]]
    free = {2, 5, 6, 9}
    slots, pos, out, status = ref.assign(table, [3, 0, 2, 4], [0, 1, 6, 9, 14], 14, free, 4)
    assert slots == [7 * 4 + 3] + [8, 9, 10, 11, 20] + [14, 15, 24] + [-1] * 5
    assert pos == [3] + [0, 1, 2, 3, 4] + [2, 3, 4] + [4, 5, 6, 7, 8]
    assert out == [4, 5, 5, 4] and status == 8 and free == {9}
    assert table == [[7, -1, -1], [2, 5, -1], [3, 6, -1], [8, -1, -1]]
    ref.release(table, [4, 0, 5, 4], free, 4)
    assert free == {9, 2, 5} and table[1] == [-1, -1, -1]


def test_rotation_by_hand():
    x = torch.zeros(1, 1, 128)
    x[0, 0, :4] = torch.tensor([1.0, 2.0, 3.0, 4.0])
    f = torch.zeros(8, dtype=torch.float64)
    f[0] = math.pi / 2  # a quarter turn a token
    y, _ = ref.rotate(x, torch.tensor([1]), f, True, 2.0)
    assert torch.allclose(y[0, 0, :4], torch.tensor([-4.0, 2.0, 6.0, 8.0], dtype=torch.float64))
    y, _ = ref.rotate(x, torch.tensor([5]), f, False, 1.0)
    assert torch.allclose(y[0, 0, [0, 1, 2, 3, 8]], torch.tensor([0.0, 2.0, 3.0, 4.0, 1.0], dtype=torch.float64))


def test_chunk_by_hand():
    """Two keys of equal score: the second row's state is their mean."""
    q = torch.zeros(2, 1, 128).half()
    k, v = torch.zeros(1, 4, 1, 128).half(), torch.zeros(1, 4, 1, 128).half()
    v[0, 0], v[0, 1] = 1.0, 3.0
    table = torch.tensor([[0]])
    o, lse, *_ = ref.chunk(q, [0, 2], k, v, table, [2], 1.0)
    assert float(o[0, 0, 5]) == 1.0 and float(o[1, 0, 5]) == 2.0
    assert float(lse[0, 0]) == 0.0 and float(lse[1, 0]) == pytest.approx(math.log(2))
    o, lse, *_ = ref.chunk(q, [0, 2], k, v, table, [1], 1.0)  # the first row stands before the first token
    assert math.isinf(float(lse[0, 0])) and float(o[1, 0, 5]) == 1.0
    o, _, *_ = ref.chunk(q, [0, 2], k, v, table, [2], 1.0, window=1)
    assert float(o[1, 0, 5]) == 3.0
