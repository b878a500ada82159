"""Attention of trees of drafts on the GPU: what weights, masks and queries may hold."""
import pytest
import torch

from tests import draft_reference as DR
from tests import fp8_reference as R
from tests.test_gpu_draft import check_tree, run_tree, seen
from tests.test_gpu_fp8 import D, DT, Setup, cu_of, i32, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,batch,new", [(1, 1, 1, 7), (8, 2, 20, 16), (16, 2, 12, 64), (20, 20, 6, 33)])
def test_tree_weights_in_calls_of_all_sizes(tq, dtype, hq, hkv, batch, new):  # noqa: F811
    """7 to 12288 query rows: a weight is off by 2^-17 of itself and no more in any row of any of them (both parts rounded
    to bf16, 2^-9 * 2^-9, and the sum's fp32 roundings in proportion).  Flat scores of small queries, so that what the
    scores' own rounding moves is less than that, and values of both signs, so that many outputs are sums that cancel."""
    gen = torch.Generator().manual_seed(batch * 100 + new)
    starts = [(40, 168, 296, 936)[b % 4] for b in range(batch)]
    lens = [a + new for a in starts]
    s = Setup(tq, gen, lens, hkv, 16)
    s.fill(lens, outliers=False)
    sees = [DR.ancestors(DR.tree(new, gen)) for _ in range(batch)]
    q = (torch.randn(batch * new, hq, D, generator=gen) / 16).to(DT[dtype]).cuda()
    out, flags = run_tree(tq, s, q, starts, [new] * batch, sees, 1)
    assert flags == 0
    for b, a in enumerate(starts):
        k, v = R.stored(s.pool, s.scales, s.rows[b], a + new)
        rows = slice(b * new, (b + 1) * new)
        check_tree(out[rows], q[rows], k, v, seen(a, sees[b]), weights=2.0 ** -17)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tree_rows_of_no_sequence_change_no_byte(tq, dtype):  # noqa: F811
    """A call padded to more rows, as a captured one is: the rows that belong to sequences keep their bytes."""
    gen = torch.Generator().manual_seed(3)
    starts, news, hq = [40, 900], [16, 20], 8
    lens = [a + n for a, n in zip(starts, news)]
    s = Setup(tq, gen, lens, 2, 16)
    s.fill(lens, outliers=False)
    sees = [DR.ancestors(DR.tree(n, gen)) for n in news]
    T, more = sum(news), 400
    q = torch.randn(T + more, hq, D, generator=gen).to(DT[dtype]).cuda()
    mask = torch.cat((DR.mask_words(sees, 1), torch.full((more, 1), -1))).cuda()
    alone = s.cache.tree(q[:T], i32(cu_of(news)), i32(starts), s.table, mask[:T].contiguous())
    out = torch.full((T + more, hq, D), 7.0, dtype=DT[dtype], device="cuda")
    s.cache.tree(q, i32(cu_of(news)), i32(starts), s.table, mask, out=out)
    assert torch.equal(out[:T], alone) and (out[T:] == 7).all()
