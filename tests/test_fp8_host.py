"""Refusals and host logic of the 8-bit paged cache's calls, without a GPU: every argument is checked before the
first CUDA call, so made-up pointers do."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def tq():
    from online_kv_cache_encode_gb300 import build
    build.build()
    from online_kv_cache_encode_gb300 import tq as T
    return T


@pytest.fixture(scope="module")
def cache(tq):
    h = P()
    assert tq.lib().tq_fp8_cache_create(P(0x100000), P(0x200000), 64, 16, 4, 128, ctypes.byref(h)) == tq.TQ_OK
    yield h
    tq.lib().tq_fp8_cache_free(h)


def test_create(tq):
    L, h = tq.lib(), P()
    make = lambda pool=0x1000, sc=0x2000, nb=8, bs=16, hkv=2, d=128: L.tq_fp8_cache_create(  # noqa: E731
        P(pool), P(sc), nb, bs, hkv, d, ctypes.byref(h))
    assert L.tq_fp8_cache_create(P(0x1000), P(0x2000), 8, 16, 2, 128, None) == tq.TQ_ERR_INVALID_ARG
    for bad in (dict(pool=0), dict(sc=0), dict(pool=0x1008), dict(sc=0x2004), dict(nb=0), dict(nb=-1), dict(bs=0),
                dict(hkv=0), dict(d=0)):
        assert make(**bad) == tq.TQ_ERR_INVALID_ARG, bad
        assert not h.value
    for bad in (dict(d=64), dict(bs=8), dict(bs=24), dict(bs=256), dict(hkv=1 << 17), dict(nb=1 << 26),
                dict(nb=1 << 60)):
        assert make(**bad) == tq.TQ_ERR_UNSUPPORTED, bad
        assert not h.value
    for bs in (16, 32, 64, 128):
        assert make(bs=bs) == tq.TQ_OK and h.value
        L.tq_fp8_cache_free(h)
    assert make(nb=(1 << 31) // (2 * 16 * 2) - 1) == tq.TQ_OK  # the largest pool
    L.tq_fp8_cache_free(h)
    L.tq_fp8_cache_free(None)


A = 0x10000  # an aligned address


def ragged(**k):
    d = dict(T=5, B=2, cu=A, start=A, table=A, mb=3)
    d.update(k)
    return d


BATCH = [ragged(T=-1), ragged(T=1 << 31), ragged(B=-1), ragged(cu=0), ragged(start=0), ragged(table=0), ragged(mb=0)]


def test_write(tq, cache):
    def call(h=cache, K=A, V=A, dt=1, ks=(512, 128), vs=(512, 128), r=ragged()):
        return tq.lib().tq_fp8_write(h, P(K), P(V), dt, *ks, *vs, r["T"], r["B"], P(r["cu"]), P(r["start"]),
                                     P(r["table"]), r["mb"], None, None)
    for r in BATCH:
        assert call(r=r) == tq.TQ_ERR_INVALID_ARG, r
    assert call(h=None) == tq.TQ_ERR_INVALID_ARG
    for k in (dict(K=0), dict(V=0), dict(K=A + 8), dict(V=A + 2), dict(dt=7), dict(ks=(-512, 128)),
              dict(ks=(516, 128)), dict(vs=(512, 132)), dict(vs=(512, -8)), dict(dt=0, ks=(514, 128))):
        assert call(**k) == tq.TQ_ERR_INVALID_ARG, k
    assert tq.lib().tq_last_error()
    assert call(r=ragged(B=(1 << 31) - 1)) == tq.TQ_ERR_UNSUPPORTED
    assert call(r=ragged(T=0, cu=0)) == tq.TQ_OK and call(r=ragged(B=0, cu=0)) == tq.TQ_OK


def test_read(tq, cache):
    def call(h=cache, K=A, V=A, dt=1, r=ragged()):
        return tq.lib().tq_fp8_read(h, P(K), P(V), dt, r["T"], r["B"], P(r["cu"]), P(r["start"]), P(r["table"]),
                                    r["mb"], None, None)
    for r in BATCH:
        assert call(r=r) == tq.TQ_ERR_INVALID_ARG, r
    for k in (dict(h=None), dict(K=0), dict(V=0), dict(K=A + 8), dict(dt=-1)):
        assert call(**k) == tq.TQ_ERR_INVALID_ARG, k
    assert call(r=ragged(B=(1 << 31) - 1)) == tq.TQ_ERR_UNSUPPORTED
    assert call(r=ragged(T=0, cu=0)) == tq.TQ_OK


ATTN = [(dict(q=0), "INVALID_ARG"), (dict(out=0), "INVALID_ARG"), (dict(ws=0), "INVALID_ARG"),
        (dict(q=A + 8), "INVALID_ARG"), (dict(out=A + 8), "INVALID_ARG"), (dict(ws=A + 16), "INVALID_ARG"),
        (dict(qs=(1028, 128)), "INVALID_ARG"), (dict(qs=(1024, -128)), "INVALID_ARG"), (dict(hq=6), "INVALID_ARG"),
        (dict(hq=0), "INVALID_ARG"), (dict(dt=5), "INVALID_ARG"), (dict(dt=0), "UNSUPPORTED"),
        (dict(hq=4 * 129), "UNSUPPORTED"), (dict(sm=0.0), "INVALID_ARG"), (dict(sm=-1.0), "INVALID_ARG"),
        (dict(sm=float("nan")), "INVALID_ARG"), (dict(sm=float("inf")), "INVALID_ARG"), (dict(nws=16), "WORKSPACE"),
        (dict(h=None), "INVALID_ARG")]


def test_decode(tq, cache):
    def call(h=cache, q=A, dt=1, qs=(1024, 128), B=2, hq=8, table=A, mb=3, lens=A, sm=0.1, out=A, ws=A, nws=1 << 30):
        return tq.lib().tq_fp8_decode_attention(h, P(q), dt, *qs, B, hq, P(table), mb, P(lens), sm, P(out), P(ws), nws,
                                                None, None)
    for k, e in ATTN + [(dict(table=0), "INVALID_ARG"), (dict(lens=0), "INVALID_ARG"), (dict(mb=0), "INVALID_ARG"),
                        (dict(B=-1), "INVALID_ARG"), (dict(B=1 << 25, mb=1 << 12), "UNSUPPORTED"),
                        (dict(B=(1 << 31) - 1, mb=(1 << 31) - 1, nws=1 << 60), "UNSUPPORTED")]:
        assert call(**k) == getattr(tq, "TQ_ERR_" + e), k
    assert call(B=0, q=0) == tq.TQ_OK
    L = tq.lib()
    assert L.tq_fp8_decode_workspace_bytes(None, 1, 4) == 0 and L.tq_fp8_decode_workspace_bytes(cache, 0, 4) == 0
    assert L.tq_fp8_decode_workspace_bytes(cache, 1, 6) == 0 and L.tq_fp8_decode_workspace_bytes(cache, 1, 4) > 0


def test_prefill(tq, cache):
    def call(h=cache, q=A, dt=1, qs=(1024, 128), hq=8, sm=0.1, out=A, ws=A, nws=1 << 30, r=ragged()):
        return tq.lib().tq_fp8_prefill_attention(h, P(q), dt, *qs, r["T"], r["B"], hq, P(r["cu"]), P(r["start"]),
                                                 P(r["table"]), r["mb"], sm, P(out), P(ws), nws, None, None)
    for k, e in ATTN:
        assert call(**k) == getattr(tq, "TQ_ERR_" + e), k
    for r in BATCH:
        assert call(r=r) == tq.TQ_ERR_INVALID_ARG, r
    assert call(r=ragged(B=(1 << 31) - 1), nws=1 << 60) == tq.TQ_ERR_UNSUPPORTED
    assert call(r=ragged(T=0, cu=0)) == tq.TQ_OK
    L = tq.lib()
    assert L.tq_fp8_prefill_workspace_bytes(cache, 0, 1, 4) == 0 and L.tq_fp8_prefill_workspace_bytes(cache, 9, 0, 4) == 0
    assert L.tq_fp8_prefill_workspace_bytes(cache, 9, 1, 5) == 0 and L.tq_fp8_prefill_workspace_bytes(cache, 9, 1, 4) > 0


def test_calls_without_a_device_refuse(tq, cache):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is there")
    r = ragged()
    assert tq.lib().tq_fp8_write(cache, P(A), P(A), 1, 512, 128, 512, 128, r["T"], r["B"], P(A), P(A), P(A), 3, None,
                                 None) == tq.TQ_ERR_CUDA
