"""The layout of the 8-bit cache's decode workspace, without a GPU: counters that have to be zero lie behind partials of
any contents, at an offset that no call's sizes change."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def tq():
    from online_kv_cache_encode_gb300 import build
    build.build()
    from online_kv_cache_encode_gb300 import tq as T
    return T


@pytest.mark.parametrize("hkv", [1, 8])
def test_counters_lie_behind_the_partials(tq, hkv):
    L, h = tq.lib(), P()
    assert L.tq_fp8_cache_create(P(0x100000), P(0x200000), 64, 16, hkv, 128, ctypes.byref(h)) == tq.TQ_OK
    at = L.tq_fp8_decode_counters_offset(h)
    assert at > 0 and at % 256 == 0
    for batch in (1, 3, 64, 1000):
        for group in (1, 8, 9, 40, 128):
            items = batch * hkv * (1 if group <= 8 else -(-group // 16))
            behind = L.tq_fp8_decode_workspace_bytes(h, batch, hkv * group) - at
            assert 4 * items <= behind < 4 * items + 256
    L.tq_fp8_cache_free(h)
    assert L.tq_fp8_decode_counters_offset(None) == 0
