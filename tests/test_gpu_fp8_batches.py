"""The 8-bit paged cache on the GPU: very large batches, and scales of the scores."""
import pytest
import torch

from tests import fp8_reference as R
from tests.test_gpu_fp8 import D, DECODE, DT, PREFILL, Setup, check, cu_of, i32, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,step", [(1100, 1), (2100, 7), (2100, 67)])
def test_batches_of_thousands(tq, batch, step):  # noqa: F811
    """More sequences than two rounds of the look-up hold, with new tokens in every one, in every seventh, and between
    runs of 66 empty ones; a long tail of empty ones, and rows behind it."""
    gen = torch.Generator().manual_seed(batch + step)
    hkv, bs = 2, 16
    news = [0 if b % step or b > batch - 90 else 1 + (b // step % 5 == 2) * 20 for b in range(batch)]
    starts = torch.randint(0, 40, (batch,), generator=gen).tolist()
    lens = [a + n for a, n in zip(starts, news)]
    s = Setup(tq, gen, lens, hkv, bs)
    T = sum(news)
    K, V = (torch.randn(sum(lens), hkv, D, generator=gen).bfloat16() for _ in range(2))
    s.cache.write(K.cuda(), V.cuda(), i32(cu_of(lens)), i32([0] * batch), s.table)
    pool, scales = s.pool.cpu(), s.scales.cpu()
    some = [b for b in range(batch) if news[b]][::37] + [0, batch - 1]
    for b in some:                       # the long write is right by sample, the short one below by every byte
        at = cu_of(lens)[b]
        p, _ = R.write(pool, scales, K[at:at + lens[b]], V[at:at + lens[b]], [0, lens[b]], [0], [s.rows[b]])
        assert torch.equal(p, pool)
    cu, st = i32(cu_of(news)), tq.new_status()
    X, Y = (torch.randn(T + 3, hkv, D, generator=gen).bfloat16() for _ in range(2))
    want = R.write(pool, scales, X, Y, cu_of(news), starts, s.rows)
    s.cache.write(X.cuda(), Y.cuda(), cu, i32(starts), s.table, status=st)
    assert torch.equal(s.pool.cpu(), want[0])
    assert torch.equal(s.scales.cpu().view(torch.int32), want[1].view(torch.int32))
    back = tuple(torch.full((T + 3, hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s.cache.read(cu, i32(starts), s.table, T + 3, out=back, status=st)
    q = torch.randn(T + 3, 4, D, generator=gen).bfloat16().cuda()
    out = torch.full_like(q, 7)
    s.cache.prefill(q, cu, i32(starts), s.table, out=out, status=st)
    one = s.cache.decode(q[:1].repeat(batch, 1, 1), s.table, i32(lens), status=st)
    assert st.item() == 0 and all((x[T:] == 7).all() for x in (out, *back))
    at = 0
    for b, (a, n) in enumerate(zip(starts, news)):
        if n or b % 50 == 0:
            k, v = R.stored(s.pool, s.scales, s.rows[b], a + n)
            check(one[b:b + 1], q[:1], k, v, [a + n], DECODE)
        if n:
            check(out[at:at + n], q[at:at + n], k, v, [a + i + 1 for i in range(n)], PREFILL)
            for x, y in zip(back, (k, v)):
                assert torch.equal(x[at:at + n], y[:, a:].permute(1, 0, 2).to(torch.bfloat16))
        at += n


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sm_scale", [0.5, 0.01, 2.0 ** -20])
def test_scale_of_the_scores(tq, dtype, sm_scale):  # noqa: F811
    gen = torch.Generator().manual_seed(72)
    n, new = 700, 50
    s = Setup(tq, gen, [n], 2, 32)
    s.fill([n], outliers=False)
    q = torch.randn(new, 6, D, generator=gen).to(DT[dtype]).cuda()
    k, v = R.stored(s.pool, s.scales, s.rows[0], n)
    out = s.cache.prefill(q, i32([0, new]), i32([n - new]), s.table, sm_scale=sm_scale)
    check(out, q, k, v, [n - new + i + 1 for i in range(new)], PREFILL, sm_scale)
    out = s.cache.decode(q[:1], s.table, i32([n]), sm_scale=sm_scale)
    check(out, q[:1], k, v, [n], DECODE, sm_scale)
