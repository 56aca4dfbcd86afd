"""Refusals of the compressed, bounded cache's entry points, without a GPU:
bad arguments are rejected before any device work."""
import ctypes

import numpy as np
import pytest
import torch

import mx4_reference as ref
import paged_kv_cascade_gb300 as pkc
from paged_kv_cascade_gb300 import build as pkc_build

F, WS = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x100000)
OFF = ctypes.c_void_p(0x1008)  # 8-byte aligned only
OFF2 = ctypes.c_void_p(0x1002)


@pytest.fixture(scope="module")
def L():
    pkc_build.build()
    return pkc.lib()


def variants(good, changes):
    """(position, value, expected code) applied one at a time to the good arguments."""
    for pos, val, code in changes:
        yield good[:pos] + [val] + good[pos + 1:], code


def test_append_mx4_refuses(L):
    # k_new v_new indptr total | kc ks vc vs | table stride lens | batch hkv d ps pages dtype ws bytes stream
    good = [F, F, F, 4, F, F, F, F, F, 4, F, 2, 8, 128, 16, 10, 1, WS, 1 << 20, None]
    for args, code in variants(good, [
            (0, None, 1), (1, None, 1), (2, None, 1), (4, None, 1), (5, None, 1), (8, None, 1), (10, None, 1),
            (0, OFF, 1), (4, OFF, 1), (6, OFF, 1), (5, OFF2, 1), (3, -1, 1), (9, 0, 1), (11, -1, 1), (12, 0, 1),
            (13, 64, 2), (14, 0, 1), (15, -1, 1), (16, 0, 1), (16, 3, 1), (17, None, 3), (17, F, 3), (18, 16, 3)]):
        if code == 3 and args[17] is F:
            args[17] = ctypes.c_void_p(0x100010)
        assert L.pkc_append_kv_mx4(*args) == code, (args, L.pkc_last_error())
    assert L.pkc_append_kv_mx4(*good[:3], 0, *good[4:]) == 0   # no rows
    assert L.pkc_append_kv_mx4(*good[:11], 0, *good[12:]) == 0  # no requests


def test_gather_mx4_refuses(L):
    # kc ks vc vs | table stride first indptr | total batch hkv d ps pages | k v dtype ws bytes stream
    good = [F, F, F, F, F, 4, F, F, 4, 2, 8, 128, 16, 10, F, F, 1, WS, 1 << 20, None]
    for args, code in variants(good, [
            (0, None, 1), (3, None, 1), (4, None, 1), (6, None, 1), (7, None, 1), (14, None, 1), (15, None, 1),
            (14, OFF, 1), (2, OFF, 1), (3, OFF2, 1), (5, 0, 1), (8, -2, 1), (11, 256, 2), (12, -4, 1), (16, 3, 1),
            (18, 255, 3)]):
        assert L.pkc_gather_kv_mx4(*args) == code, (args, L.pkc_last_error())
    assert L.pkc_gather_kv_mx4(*good[:8], 0, *good[9:]) == 0


def test_decode_mx4_refuses(L):
    # q kc ks vc vs | table stride lens | batch hq hkv d ps pages scale plan ws bytes o lse dtype stream
    good = [F, F, F, F, F, F, 4, F, 2, 16, 8, 128, 16, 10, 1.0, None, WS, 1 << 20, F, F, 1, None]
    for args, code in variants(good, [
            (0, None, 1), (1, None, 1), (4, None, 1), (5, None, 1), (7, None, 1), (18, None, 1), (19, None, 1),
            (0, OFF, 1), (1, OFF, 1), (2, OFF2, 1), (18, OFF, 1), (6, 0, 1), (9, 12, 1), (9, 24, 2), (11, 64, 2),
            (12, 0, 1), (13, -1, 1), (20, 0, 1), (17, 300, 3)]):
        assert L.pkc_paged_decode_state_mx4(*args) == code, (args, L.pkc_last_error())
    plan = pkc.plan([5, 6, 7], 4)  # of another batch
    args = good[:15] + [ctypes.c_void_p(plan.ctypes.data)] + good[16:]
    assert L.pkc_paged_decode_state_mx4(*args) == 7
    assert L.pkc_paged_decode_state_mx4(*good[:8], 0, *good[9:]) == 0


def test_binding_refuses_host_tensors():
    u8 = torch.uint8
    pools = [torch.zeros(4, 16, 2, n, dtype=u8) for n in (64, 4, 64, 4)]
    bt, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ip, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(1024, dtype=u8)
    x, q = torch.zeros(2, 2, 128).half(), torch.zeros(2, 4, 128).half()
    with pytest.raises(ValueError, match="CUDA"):
        pkc.append_kv_mx4(x, x, ip, *pools, bt, lens, ws)
    with pytest.raises(ValueError, match="CUDA"):
        pkc.gather_kv_mx4(*pools, bt, lens, ip, 2, ws)
    with pytest.raises(ValueError, match="CUDA"):
        pkc.paged_decode_state_mx4(q, *pools, bt, lens, 0.1, ws)
    with pytest.raises(ValueError, match="shape"):
        pkc.paged_decode_state_mx4(q, pools[1], *pools[1:], bt, lens, 0.1, ws)
    with pytest.raises(TypeError, match="dtype"):
        pkc.paged_decode_state_mx4(q, pools[0].to(torch.int32), *pools[1:], bt, lens, 0.1, ws)


def test_mx4_reference_is_the_nearest_code():
    """The reference's own pins: hand-computed blocks, ties, saturation, zeros."""
    x = np.zeros((1, 128))
    x[0, :8] = [6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]
    x[0, 32:36] = [7.9, -7.1, 0.24, -0.26]
    x[0, 64] = 2.0 ** -140
    x[0, 96] = np.inf
    c, s = ref.quantise(x)
    v = ref.values(c, s)
    assert v[0, :8].tolist() == [6.0, 4.0, 4.0, 2.0, 2.0, 1.0, 1.0, 0.0]
    assert v[0, 32:36].tolist() == [6.0, -6.0, 0.0, -0.5]
    assert v[0, 64] == 0.0 and np.all(np.isnan(v[0, 96:]))
    assert s[0].tolist() == [127, 127, 1, 255]
    assert np.all(c.reshape(1, 8, 4, 2)[:, :, 3] == 0)  # a NaN block's codes


def test_accumulate_weights_refuses(L):
    # q lse k ks table stride lens | batch hq hkv d ps pages sm k_scale decay w W dtype kv ws bytes stream
    good = [F, F, F, None, F, 4, F, 2, 16, 8, 128, 16, 10, 1.0, 1.0, 1.0, F, 64, 1, 1, WS, 1 << 20, None]
    nan, inf = float("nan"), float("inf")
    for args, code in variants(good, [
            (0, None, 1), (1, None, 1), (2, None, 1), (4, None, 1), (6, None, 1), (16, None, 1), (0, OFF, 1),
            (2, OFF, 1), (5, 0, 1), (7, -1, 1), (8, 12, 1), (8, 24, 2), (10, 64, 2), (11, 0, 1), (11, 1 << 30, 2),
            (12, -1, 1), (14, 0.0, 1), (14, 2.0, 1), (14, nan, 1), (15, -0.5, 1), (15, 1.5, 1), (15, nan, 1),
            (15, inf, 1), (17, 0, 1), (18, 2, 1), (18, 0, 1), (19, 2, 1), (19, 0, 1), (19, 5, 1), (19, 4, 1),
            (21, 100, 3)]):
        assert L.pkc_accumulate_weights(*args) == code, (args, L.pkc_last_error())
    # an e4m3 cache takes fp16 queries and a finite scale > 0
    for args, code in variants(good[:19] + [3] + good[20:], [(18, 2, 1), (14, -1.0, 1), (14, inf, 1)]):
        assert L.pkc_accumulate_weights(*args) == code
    assert L.pkc_accumulate_weights(*good[:7], 0, *good[8:]) == 0


def test_evict_select_refuses(L):
    # w W lens batch hkv budget sinks recent keep ws bytes stream
    good = [F, 64, F, 2, 8, 16, 4, 8, F, WS, 1 << 20, None]
    for args, code in variants(good, [
            (0, None, 1), (2, None, 1), (8, None, 1), (1, 0, 1), (3, -1, 1), (4, 0, 1), (5, 0, 1), (5, 11, 1),
            (6, -1, 1), (7, -1, 1), (7, 13, 1), (6, 2 ** 31 - 1, 1), (5, 2 ** 30 + 1, 2), (3, 1 << 28, 2), (10, 255, 3)]):
        assert L.pkc_evict_select(*args) == code, (args, L.pkc_last_error())
    assert L.pkc_evict_select(*good[:3], 0, *good[4:]) == 0


def test_evict_compact_refuses(L):
    # keep budget k v ks vs table stride lens w W | batch hkv d ps pages kv ws bytes stream
    good = [F, 16, F, F, None, None, F, 4, F, F, 64, 2, 8, 128, 16, 10, 1, WS, 1 << 20, None]
    for args, code in variants(good, [
            (0, None, 1), (2, None, 1), (3, None, 1), (6, None, 1), (8, None, 1), (1, 0, 1), (2, OFF, 1), (3, OFF, 1),
            (7, 0, 1), (1, 2 ** 30 + 1, 2), (10, 0, 1), (11, -1, 1), (11, 1 << 26, 2), (12, 0, 1), (13, 64, 2), (14, 0, 1), (15, -1, 1),
            (16, 0, 1), (16, 5, 1), (16, 4, 1), (18, 200, 3)]):
        assert L.pkc_evict_compact(*args) == code, (args, L.pkc_last_error())
    assert L.pkc_evict_compact(*good[:11], 0, *good[12:]) == 0


def test_eviction_binding_refuses_before_any_call():
    w, lens = torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int32)
    bt, ws = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(1024, dtype=torch.uint8)
    k = torch.zeros(4, 16, 2, 128).half()
    with pytest.raises(ValueError, match="CUDA"):
        pkc.evict_select(w, lens, 8, 1, 1, ws)
    with pytest.raises(ValueError, match="CUDA"):
        pkc.accumulate_weights(torch.zeros(2, 4, 128).half(), torch.zeros(2, 4), k, bt, lens, 0.1, w, ws)
    with pytest.raises(ValueError, match="CUDA"):
        pkc.evict_compact(torch.zeros(2, 2, 8, dtype=torch.int32), k, k, bt, lens, ws)
    with pytest.raises(TypeError, match="dtype"):
        pkc.evict_compact(torch.zeros(2, 2, 8, dtype=torch.int32), k.float(), k, bt, lens, ws)
