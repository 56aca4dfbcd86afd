"""Sizes that the compressed, bounded cache's entry points cannot launch, on
the CPU: an error code comes back.  In a process of its own, as what is
refused here could otherwise end or hold the process."""
import subprocess
import sys

import pytest

from conftest import ROOT

HEAD = """
import ctypes
import paged_kv_cascade_gb300 as pkc
from paged_kv_cascade_gb300 import build
build.build()
L, F, WS = pkc.lib(), ctypes.c_void_p(0x1000), ctypes.c_void_p(0x100000)
"""


def code_of(call):
    r = subprocess.run([sys.executable, "-c", HEAD + f"print('code', {call})"], cwd=ROOT, capture_output=True, text=True,
                       timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    return int(r.stdout.split("code")[-1])


@pytest.mark.parametrize("batch,hq,hkv", [(2 ** 31 - 1, 8, 8), (2 ** 30, 64, 64), (2 ** 31 - 1, 2 ** 16, 2 ** 16)])
def test_weights_of_more_rows_than_a_grid_has_blocks(batch, hq, hkv):
    # q lse k ks table stride lens | batch hq hkv d ps pages sm k_scale decay w W dtype kv ws bytes stream
    call = (f"L.pkc_accumulate_weights(F, F, F, None, F, 4, F, {batch}, {hq}, {hkv}, 128, 16, 10, 1.0, 1.0, 1.0, F, 64, "
            "1, 1, WS, 1 << 20, None)")
    assert code_of(call) == 2


@pytest.mark.parametrize("call", [
    "L.pkc_append_kv_mx4(F, F, F, 4, F, F, F, F, F, 4, F, 2, {hkv}, 128, 16, 10, 1, WS, 1 << 20, None)",
    "L.pkc_gather_kv_mx4(F, F, F, F, F, 4, F, F, 4, 2, {hkv}, 128, 16, 10, F, F, 1, WS, 1 << 20, None)",
    "L.pkc_accumulate_weights(F, F, F, None, F, 4, F, 2, {hkv}, {hkv}, 128, 16, 10, 1.0, 1.0, 1.0, F, 64, 1, 1, WS, 1 << 20, None)",
    "L.pkc_evict_compact(F, 16, F, F, None, None, F, 4, F, F, 64, 2, {hkv}, 128, 16, 10, 1, WS, 1 << 20, None)",
])
@pytest.mark.parametrize("hkv", [2 ** 16 + 1, 2 ** 25, 2 ** 30 + 1])
def test_more_heads_than_a_row_can_be_addressed_with(call, hkv):
    """A token's heads lie within 2^32 bytes and a grid's second dimension."""
    assert code_of(call.format(hkv=hkv)) == 2
