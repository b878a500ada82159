"""Attention of trees of drafts on the GPU: what weights, masks and queries may hold."""
import math

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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,new", [(1, 100), (4, 30), (2, 100), (8, 16)])   # of one row tile and of two
@pytest.mark.parametrize("start", [0, 284])
@pytest.mark.parametrize("steps", [(0, 26, 52, 80), (0, 0, 32, 0), (80, 0, 0, 80), (0, 32, 0, 64)])
def test_tree_references_raised_within_a_tile(tq, dtype, hq, new, start, steps):  # noqa: F811
    """Scores that rise by tens of octaves from one 32 tokens of a tile to the next, and rows that see their first token
    in any of them, so that weights that are already formed are scaled again, in some rows of a warp and not in others;
    values as large as the weights are small, so that every weight counts in the output."""
    gen = torch.Generator().manual_seed(hq + sum(steps))
    n = start + new
    s = Setup(tq, gen, [n], 1, 16)
    # dim 0 carries the step of a token's 32 (halves of the steps are exact in e4m3): with 16 in a query's dim 0 its
    # score is that many octaves, and the product of weight and value about 1
    step = torch.tensor(steps, dtype=torch.float32)[torch.arange(n) % 128 // 32]
    K, V = torch.randn(n, 1, D, generator=gen) / 4, torch.randn(n, 1, D, generator=gen)
    K[:, 0, 0] = step / 2
    V *= torch.exp2(80 - step)[:, None, None]
    p, sc = R.write(s.pool.cpu(), s.scales.cpu(), K, V, [0, n], [0], s.rows)
    s.pool.copy_(p)
    s.scales.copy_(sc)
    most = float(step.max())
    if dtype == "f16":   # (outputs within the type's range)
        s.scales[:, :, 1] *= 2.0 ** (most - 80)
    q = torch.randn(new, hq, D, generator=gen)
    q[..., 0] = torch.tensor([16.0, 8.0, 20.0, 0.0] if dtype == "bf16" else [16.0, 20.0, 16.0, 24.0])[torch.arange(new) % 4][:, None]
    q = q.to(DT[dtype]).cuda()
    see = DR.ancestors(DR.tree(new, gen))
    if start == 0 and dtype == "f16":   # (a row that sees no token of the largest step would be past it)
        see[:, int(step.argmax())] = True
    sm_scale = math.log(2) / 8
    out, flags = run_tree(tq, s, q, [start], [new], [see], 2, sm_scale=sm_scale)
    assert flags == 0
    k, v = R.stored(s.pool, s.scales, s.rows[0], n)
    check_tree(out, q, k, v, seen(start, see), sm_scale, weights=2.0 ** -17)
    assert torch.equal(run_tree(tq, s, q, [start], [new], [see], 2, sm_scale=sm_scale)[0], out)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq", [1, 8, 60])
def test_tree_nonfinite_queries_that_see_nothing(tq, dtype, hq):  # noqa: F811
    """A row that attends to nothing is zero whatever its query holds (a padded step's rows may hold anything): by its
    mask, by a negative start, by blocks that are not there; one that sees a token is NaN, also where the unit is cut and
    where it sees nothing in most of the tiles; the others keep their bytes."""
    gen = torch.Generator().manual_seed(hq)
    starts, news = [0, -7, 20, 3000], [300, 9, 12, 40]
    lens = [max(a, 0) + n for a, n in zip(starts, news)]
    s = Setup(tq, gen, lens, 1, 16)
    s.fill(lens)
    table = s.table.clone()
    table[2, :3] = -1
    sees = [DR.ancestors(DR.tree(n, gen)) for n in news]
    sees[0][::3] = False
    sees[0][9, 290] = sees[0][12, 3] = True      # one token, in the last tile and in the first
    q = torch.randn(sum(news), hq, D, generator=gen).to(DT[dtype]).cuda()
    cu, mask = cu_of(news), DR.mask_words(sees, 5).cuda()
    good = s.cache.tree(q, i32(cu), i32(starts), table, mask)
    bad = q.clone()
    spoilt = torch.zeros(sum(news), hq, dtype=torch.bool)
    for row, x in ((0, math.nan), (3, math.inf), (6, -math.inf), (9, math.nan), (12, math.inf), (5, math.nan), (299, math.inf), (301, math.nan),
                   (305, math.inf), (310, math.nan), (320, -math.inf), (330, math.nan), (331, math.inf)):
        spoilt[row, row % hq] = True
        bad[row, row % hq, row % D] = x
    st = tq.new_status()
    out = s.cache.tree(bad, i32(cu), i32(starts), table, mask, status=st)
    assert st.item() == tq.FLAG_BAD_SLOT
    nothing = torch.cat((~sees[0].any(1), torch.ones(9 + 12, dtype=torch.bool), torch.zeros(40, dtype=torch.bool)))
    assert not out[nothing.cuda()].any() and not good[nothing.cuda()].any()
    nan = spoilt & ~nothing[:, None]
    assert torch.isnan(out[nan.cuda()]).all() and nan.sum() == 6
    assert torch.equal(out[~nan.cuda()], good[~nan.cuda()])
