"""Refusals and host logic of the operators for drafted tokens, without a GPU: every argument is checked before the
first CUDA call, so made-up pointers do."""
import ctypes
import math

import numpy as np
import pytest

from tests import draft_reference as DR
from tests.test_fp8_host import A, ATTN, BATCH, P, cache, ragged, tq  # noqa: F401

INVALID, UNSUPPORTED = "INVALID_ARG", "UNSUPPORTED"
TABLE = [(dict(table=0), INVALID), (dict(table=A + 8), INVALID), (dict(far=0), INVALID), (dict(far=1 << 31), UNSUPPORTED),
         (dict(rot=0), INVALID), (dict(rot=-16), INVALID), (dict(rot=24), UNSUPPORTED), (dict(rot=272), UNSUPPORTED),
         (dict(layout=2), INVALID)]


@pytest.mark.parametrize("rot,base,scaling", [
    (128, 10000.0, None), (64, 500000.0, ("linear", 4.0)), (96, 10000.0, ("base", 8.0)),
    (128, 500000.0, ("parts", 8.0, 8192, 1.0, 4.0)), (16, 100.0, ("parts", 0.5, 100, -1.0, 0.0)), (2, 7.0, None)])
def test_frequencies(tq, rot, base, scaling):  # noqa: F811
    got = tq.rotary_frequencies(rot, base, scaling)
    np.testing.assert_allclose(got, DR.frequencies(rot, base, scaling), rtol=1e-14, atol=0)


def test_frequencies_of_a_stretched_context(tq):  # noqa: F811
    """PARTS leaves fast pairs alone and stretches slow ones; BASE moves the slowest by the factor, the fastest not."""
    plain = tq.rotary_frequencies(128, 10000.0)
    parts = tq.rotary_frequencies(128, 10000.0, ("parts", 8.0, 4096, 1.0, 32.0))
    turns = 4096 * plain / (2 * math.pi)
    assert (parts[turns >= 32] == plain[turns >= 32]).all()
    np.testing.assert_allclose(parts[turns <= 1], plain[turns <= 1] / 8, rtol=1e-15)
    between = (turns > 1) & (turns < 32)
    assert ((parts < plain) & (parts > plain / 8))[between].all() and between.any()
    based = tq.rotary_frequencies(128, 10000.0, ("base", 8.0))
    np.testing.assert_allclose([based[0], based[-1]], [plain[0], plain[-1] / 8], rtol=1e-13)


def test_frequencies_refusals(tq):  # noqa: F811
    for args in ((0, 10.0, None), (7, 10.0, None), (64, 0.0, None), (64, math.inf, None), (64, 10.0, ("linear", 0.0)),
                 (64, 10.0, ("linear", math.nan)), (2, 10.0, ("base", 2.0)), (64, 10.0, ("parts", 8.0, 0.0, 1.0, 4.0)),
                 (64, 10.0, ("parts", 8.0, 100.0, 4.0, 4.0)), (64, 10.0, ("linear",)), (64, 10.0, ("other", 1.0))):
        with pytest.raises(tq.TQError) as e:
            tq.rotary_frequencies(*args)
        assert e.value.status == tq.TQ_ERR_INVALID_ARG, args
    out = (ctypes.c_double * 32)()
    assert tq.lib().tq_rotary_frequencies(64, 10.0, 9, 1.0, 1.0, 0.0, 1.0, out) == tq.TQ_ERR_INVALID_ARG
    assert tq.lib().tq_rotary_frequencies(64, 10.0, 0, 1.0, 1.0, 0.0, 1.0, None) == tq.TQ_ERR_INVALID_ARG


def test_table(tq):  # noqa: F811
    f = (ctypes.c_double * 64)(*[1.0] * 64)

    def call(freq=f, rot=128, m=1.0, far=100, table=A):
        return tq.lib().tq_rotary_table(freq, rot, m, far, P(table), None)
    for k, e in TABLE[:-1] + [(dict(freq=None), INVALID), (dict(m=0.0), INVALID), (dict(m=-1.0), INVALID), (dict(m=math.nan), INVALID)]:
        assert call(**k) == getattr(tq, "TQ_ERR_" + e), k
    f[63] = math.inf
    assert call() == tq.TQ_ERR_INVALID_ARG


def test_rotary(tq):  # noqa: F811
    far_off = A + (1 << 30)

    def call(x=A, dt=1, xs=(1024, 128), T=5, H=8, d=128, p=A, table=A, far=100, rot=64, layout=0, out=far_off, os=(1024, 128)):
        return tq.lib().tq_rotary(P(x), dt, *xs, T, H, d, P(p), P(table), far, rot, layout, 0, P(out), *os, None, None)
    for k, e in TABLE + [(dict(x=0), INVALID), (dict(out=0), INVALID), (dict(p=0), INVALID), (dict(T=-1), INVALID),
                         (dict(H=-1), INVALID), (dict(d=0), INVALID), (dict(d=32), INVALID), (dict(d=72), UNSUPPORTED),
                         (dict(d=8192), UNSUPPORTED), (dict(dt=3), INVALID), (dict(x=A + 8), INVALID), (dict(out=far_off + 2), INVALID),
                         (dict(xs=(1028, 128)), INVALID), (dict(xs=(-1024, 128)), INVALID), (dict(os=(1024, 120)), INVALID),
                         (dict(os=(1016, 128)), INVALID), (dict(os=(0, 128)), INVALID), (dict(os=(1024, 0)), INVALID),
                         (dict(xs=(1 << 61, 128), T=9), INVALID), (dict(xs=(1 << 60, 128), T=9), INVALID),
                         (dict(out=A + 2048), INVALID), (dict(out=A, os=(2048, 128)), INVALID),
                         (dict(out=A - 1024), INVALID), (dict(dt=0, xs=(1026, 128)), INVALID),
                         (dict(T=1 << 40, xs=(0, 128), os=(1024, 128)), UNSUPPORTED)]:
        assert call(**k) == getattr(tq, "TQ_ERR_" + e), k
    assert call(T=0, x=0, out=0, p=0) == tq.TQ_OK and call(H=0, x=0) == tq.TQ_OK


def test_append(tq, cache):  # noqa: F811
    far_off = A + (1 << 30)

    def call(h=cache, K=A, V=A, dt=1, ks=(512, 128), vs=(512, 128), q=A, qs=(1024, 128), hq=8, out=far_off, os=(1024, 128),
             r=ragged(), p=None, table=A, far=100, rot=64, layout=0):
        return tq.lib().tq_fp8_append(h, P(K), P(V), dt, *ks, *vs, P(q), *qs, hq, P(out), *os, r["T"], r["B"], P(r["cu"]),
                                      P(r["start"]), P(r["table"]), r["mb"], p, P(table), far, rot, layout, None, None)
    for r in BATCH:
        assert call(r=r) == tq.TQ_ERR_INVALID_ARG, r
    for k, e in TABLE + [(dict(h=None), INVALID), (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(K=A + 8), INVALID),
                         (dict(dt=7), INVALID), (dict(ks=(-512, 128)), INVALID), (dict(vs=(512, 132)), INVALID),
                         (dict(rot=144), INVALID), (dict(out=0), INVALID), (dict(hq=0), INVALID), (dict(hq=-3), INVALID),
                         (dict(q=A + 2), INVALID), (dict(qs=(1028, 128)), INVALID), (dict(out=far_off + 8), INVALID),
                         (dict(os=(1016, 128)), INVALID), (dict(out=A + 256), INVALID),
                         (dict(r=ragged(B=(1 << 31) - 1)), UNSUPPORTED)]:
        assert call(**k) == getattr(tq, "TQ_ERR_" + e), k
    assert call(r=ragged(T=0, cu=0)) == tq.TQ_OK and call(r=ragged(B=0, cu=0)) == tq.TQ_OK


def test_tree(tq, cache):  # noqa: F811
    def call(h=cache, q=A, dt=1, qs=(1024, 128), hq=8, sm=0.1, out=A, ws=A, nws=1 << 30, r=ragged(), mask=A, words=1):
        return tq.lib().tq_fp8_tree_attention(h, P(q), dt, *qs, r["T"], r["B"], hq, P(r["cu"]), P(r["start"]), P(r["table"]),
                                              r["mb"], P(mask), words, sm, P(out), P(ws), nws, None, None)
    for k, e in ATTN + [(dict(mask=0), INVALID), (dict(mask=A + 4), INVALID), (dict(words=0), INVALID), (dict(words=-1), INVALID)]:
        assert call(**k) == getattr(tq, "TQ_ERR_" + e), k
    for r in BATCH:
        assert call(r=r) == tq.TQ_ERR_INVALID_ARG, r
    assert call(r=ragged(B=(1 << 31) - 1), nws=1 << 60) == tq.TQ_ERR_UNSUPPORTED
    assert call(r=ragged(T=0, cu=0)) == tq.TQ_OK
    L = tq.lib()
    assert L.tq_fp8_tree_workspace_bytes(cache, 0, 1, 4) == 0 and L.tq_fp8_tree_workspace_bytes(cache, 9, 0, 4) == 0
    assert L.tq_fp8_tree_workspace_bytes(None, 9, 1, 4) == 0
    assert L.tq_fp8_tree_workspace_bytes(cache, 9, 1, 5) == 0 and L.tq_fp8_tree_workspace_bytes(cache, 9, 1, 4) > 0


def test_keep(tq, cache):  # noqa: F811
    def call(h=cache, kept=A, r=ragged()):
        return tq.lib().tq_fp8_keep(h, r["T"], r["B"], P(r["cu"]), P(kept), P(r["start"]), P(r["table"]), r["mb"], None, None)
    for r in BATCH:
        assert call(r=r) == tq.TQ_ERR_INVALID_ARG, r
    assert call(h=None) == tq.TQ_ERR_INVALID_ARG and call(kept=0) == tq.TQ_ERR_INVALID_ARG
    assert call(r=ragged(T=0, cu=0)) == tq.TQ_OK


def test_mask_words_and_trees():
    """The reference's own pieces: bits of the nodes a node sees."""
    see = DR.ancestors([-1, 0, 0, 1, -1])
    assert see.tolist() == [[True, False, False, False, False], [True, True, False, False, False], [True, False, True, False, False],
                            [True, True, False, True, False], [False, False, False, False, True]]
    assert DR.mask_words([see], 1).flatten().tolist() == [1, 3, 5, 11, 16]
    import torch
    one = torch.zeros(1, 130, dtype=torch.bool)
    one[0, 63] = one[0, 64] = one[0, 129] = True
    assert DR.mask_words([one], 3).tolist() == [[-1 << 63, 1, 2]]


@pytest.mark.parametrize("dim,far,what", [(24, 10, "dims"), (0, 10, "dims"), (272, 10, "dims"), (64, 0, "positions"), (64, -1, "positions")])
def test_rotary_says_what_is_wrong(tq, dim, far, what):  # noqa: F811
    with pytest.raises(tq.TQError, match=what):
        tq.Rotary(dim, far)
