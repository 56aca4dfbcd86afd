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
