"""Drafted tokens on the GPU: calls beside other calls, sequences beside other sequences."""
import pytest
import torch

from tests import draft_reference as DR
from tests import fp8_reference as R
from tests.test_gpu_draft import check_tree, run_tree, seen
from tests.test_gpu_fp8 import D, DT, PREFILL, Setup, cu_of, i32, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,batch", [(8, 2, 40), (20, 20, 9), (4, 1, 300)])
def test_tree_rows_beside_others_and_alone(tq, dtype, hq, hkv, batch):  # noqa: F811
    """A sequence's rows in a batch and in a call of its own, where the tokens are cut into other runs: both within the
    documented rounding of the same values, and so within twice that of one another."""
    gen = torch.Generator().manual_seed(batch)
    news = torch.randint(0, 20, (batch,), generator=gen).tolist()
    starts = torch.randint(0, 700, (batch,), generator=gen).tolist()
    news[0], starts[0], news[-1] = 70, 2000, 33
    lens = [a + n if n else 0 for a, n in zip(starts, news)]
    s = Setup(tq, gen, [max(n, 1) for n in lens], hkv, 16)
    s.fill([max(n, 1) for n in lens])
    sees = [DR.ancestors(DR.tree(n, gen)) if n else torch.zeros(0, 0, dtype=torch.bool) for n in news]
    q = torch.randn(sum(news), hq, D, generator=gen).to(DT[dtype]).cuda()
    out, flags = run_tree(tq, s, q, starts, news, sees, 2)
    assert flags == 0
    cu, eps = cu_of(news), torch.finfo(DT[dtype]).eps
    some = [b for b in range(batch) if news[b]]
    for b in some[:6] + some[-6:]:
        rows = slice(cu[b], cu[b + 1])
        alone = s.cache.tree(q[rows], i32([0, news[b]]), i32([starts[b]]), s.table[b:b + 1].contiguous(), DR.mask_words([sees[b]], 2).cuda())
        k, v = R.stored(s.pool, s.scales, s.rows[b], lens[b])
        for x in (alone, out[rows]):
            check_tree(x, q[rows], k, v, seen(starts[b], sees[b]), weights=2.0 ** -17)
        want, spread, sharp = DR.attend(q[rows], k, v, seen(starts[b], sees[b]), D ** -0.5, PREFILL)
        tol = eps / 2 * want.abs() + spread * (2.0 ** -17 + 2.0 ** -19 + 2 * 2.0 ** -16 * sharp[..., None]) + 2.0 ** -25
        assert ((alone.double() - out[rows].double()).abs() <= 2 * tol).all()


def test_appends_and_keeps_beside_trees(tq):  # noqa: F811
    """One stream appends to and keeps in one sequence, step after step, while another attends to a tree of a second
    sequence of the same cache, without waiting for one another: the outputs and every byte of the pool are those of the
    calls one after the other."""
    gen = torch.Generator().manual_seed(12)
    hkv, hq, n, lens = 2, 8, 12, [500, 2900]
    setups = [Setup(tq, torch.Generator().manual_seed(5), [x + 160 for x in lens], hkv, 16) for _ in range(2)]
    for s in setups:
        s.gen = torch.Generator().manual_seed(6)
        s.fill([x + 160 for x in lens])
    r = tq.Rotary(128, 4096)
    mask = DR.mask_words([DR.ancestors(DR.tree(20, gen))], 1).cuda()
    q = torch.randn(20, hq, D, generator=gen).bfloat16().cuda()
    kept = [0, 2, 5, 9]
    steps = [(torch.randn(n, hq + 2 * hkv, D, generator=gen).bfloat16().cuda(), i32([lens[0] + i * len(kept)])) for i in range(30)]
    cu, cu_kept, places = i32([0, n]), i32([0, len(kept)]), i32(kept)
    far, cu_far = i32([lens[1]]), i32([0, 20])
    tables = [[s.table[b:b + 1].contiguous() for b in range(2)] for s in setups]

    def write(i, x, start):
        c, table = setups[i].cache, tables[i][0]
        got = c.append(x[:, hq:hq + hkv], x[:, hq + hkv:], cu, start, table, r, q=x[:, :hq])
        c.keep(cu_kept, places, start, table)
        return got

    def attend(i):
        return setups[i].cache.tree(q, cu_far, far, tables[i][1], mask)

    want_q = [write(0, *step) for step in steps]
    want = attend(0)
    attend(1)
    torch.cuda.synchronize()
    one, two, got_q, got = torch.cuda.Stream(), torch.cuda.Stream(), [], []
    for step in steps:
        with torch.cuda.stream(one):
            got_q.append(write(1, *step))
        with torch.cuda.stream(two):
            got.append(attend(1))
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for x, w in zip(got_q, want_q)) and all(torch.equal(x, want) for x in got)
    assert torch.equal(setups[0].pool, setups[1].pool)
    assert torch.equal(setups[0].scales.nan_to_num(9), setups[1].scales.nan_to_num(9))
