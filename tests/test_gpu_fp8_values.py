"""The 8-bit paged cache on the GPU: codes of NaN, values at the ends of the range, and slots that a row does not see."""
import math

import pytest
import torch

from tests import fp8_reference as R
from tests.test_gpu_fp8 import D, DECODE, DT, PREFILL, Setup, check, cu_of, i32, tq  # noqa: F401

pytestmark = pytest.mark.gpu


def clean(x):
    return torch.where(torch.isnan(x), torch.zeros_like(x), x)


def check_nan(out, q, k, v, limits, floor):
    """Row i's element d is NaN where the row sees a NaN in dim d of the values, the whole row where it sees one in the
    keys, by KV head; every other element is what it is without them."""
    group = q.shape[1] // k.shape[0]
    see = torch.arange(k.shape[1], device=q.device)[None, :] < torch.as_tensor(limits, device=q.device)[:, None]
    nan = (see[:, None, :, None] & (torch.isnan(v) | torch.isnan(k).any(-1, keepdim=True))[None]).any(2)
    nan = nan.repeat_interleave(group, 1)
    assert torch.equal(torch.isnan(out), nan)
    want = R.attend(q, clean(k), clean(v), limits, 1 / math.sqrt(D), None, floor)[0]
    check(torch.where(nan, want.to(out.dtype), out), q, clean(k), clean(v), limits, floor)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bs,hq,hkv,start,new", [
    (16, 8, 2, 0, 420),      # a unit sees the tokens that others of its rows do not
    (64, 5, 1, 2900, 7),     # the tokens split among many CTAs
    (32, 20, 20, 130, 150),
])
def test_nan_codes(tq, dtype, bs, hq, hkv, start, new):  # noqa: F811
    """A pool that another program filled may hold codes of NaN at positions that are read: they are NaN to every call,
    in the rows that see them and in no others."""
    gen = torch.Generator().manual_seed(61)
    n = start + new
    s = Setup(tq, gen, [n], hkv, bs)
    s.fill([n])
    last = [n - 1 - x for x in (0, 1, 5, new // 2, new - 1) if x < new]
    for i, p in enumerate(last + [start // 2, start // 3 + 17]):
        blk = s.rows[0][p // bs]
        s.pool[blk, 0, 1, p % bs, (37 * i + 3) % D] = 0x7F if i % 2 else 0xFF
        if i == 3:
            s.pool[blk, hkv - 1, 1, p % bs, 64:80] = 0x7F
    if hkv > 1:
        p = start + new // 3
        s.pool[s.rows[0][p // bs], 1, 0, p % bs, 9] = 0x7F
    q = torch.randn(new, hq, D, generator=gen).to(DT[dtype]).cuda()
    k, v = R.stored(s.pool, s.scales, s.rows[0], n)
    out = s.cache.prefill(q, i32([0, new]), i32([start]), s.table)
    check_nan(out, q, k, v, [start + i + 1 for i in range(new)], PREFILL)
    lens = [n, start + 1, n - 2]
    out = s.cache.decode(q[:3], s.table.repeat(3, 1), i32(lens))
    check_nan(out, q[:3], k, v, lens, DECODE)
    got = s.cache.read(i32([0, n]), i32([0]), s.table, n, torch.float32)
    for x, want in zip(got, (k, v)):
        assert torch.equal(torch.nan_to_num(x.double(), nan=7e7), torch.nan_to_num(want.permute(1, 0, 2), nan=7e7))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_nan_codes_that_no_row_sees(tq, dtype):  # noqa: F811
    """Codes of NaN behind the sequence's end, in blocks that the table does not name and in the other sequence's."""
    gen = torch.Generator().manual_seed(62)
    starts, news = [0, 77], [133, 200]
    lens = [a + b for a, b in zip(starts, news)]
    s = Setup(tq, gen, lens, 2, 16)
    s.fill(lens)
    for b, n in enumerate(lens):
        s.pool[s.rows[b][n // 16], :, :, n % 16:] = 0x7F
    s.pool[s.free] = 0xFF
    s.pool[s.rows[0][3], 1, 1, 5, 8] = 0x7F      # position 53 of sequence 0
    q = torch.randn(sum(news), 4, D, generator=gen).to(DT[dtype]).cuda()
    out = s.cache.prefill(q, i32(cu_of(news)), i32(starts), s.table)
    one = s.cache.decode(q[:2], s.table, i32(lens))
    for b, (a, n) in enumerate(zip(starts, news)):
        at = cu_of(news)[b]
        k, v = R.stored(s.pool, s.scales, s.rows[b], a + n)
        check_nan(out[at:at + n], q[at:at + n], k, v, [a + i + 1 for i in range(n)], PREFILL)
        check_nan(one[b:b + 1], q[b:b + 1], k, v, [a + n], DECODE)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("call", ["decode", "prefill"])
@pytest.mark.parametrize("octaves", [5, 7, 14, 30, 80])
@pytest.mark.parametrize("bs,hq", [(16, 3), (64, 12)])
def test_large_scales_over_codes_of_zero(tq, dtype, call, octaves, bs, hq):  # noqa: F811
    """Blocks with a few values 2^octaves the others' size, whose other values round to 0: in those dims only the other
    blocks count, though every token has its part of the weight."""
    gen = torch.Generator().manual_seed(65)
    n = 1100
    s = Setup(tq, gen, [n], 1, bs)
    K, V = (torch.randn(n, 1, D, generator=gen) for _ in range(2))
    for t in (3, 70, 71, 400, 520, 900, n - 1):
        V[t, 0, t % 7::29] *= 2.0 ** octaves
    p, sc = R.write(s.pool.cpu(), s.scales.cpu(), K, V, [0, n], [0], s.rows)
    s.pool.copy_(p)
    s.scales.copy_(sc)
    q = torch.randn(2, hq, D, generator=gen).to(DT[dtype]).cuda()
    k, v = R.stored(s.pool, s.scales, s.rows[0], n)
    lens = [n - 1, n]
    if call == "decode":
        out = s.cache.decode(q, s.table.repeat(2, 1), i32(lens))
    else:
        out = s.cache.prefill(q, i32([0, 2]), i32([n - 2]), s.table)
    floor, most = DECODE if call == "decode" else PREFILL, torch.finfo(out.dtype).max
    want = R.attend(q, k, v, lens, 1 / math.sqrt(D), None, floor)[0]
    over = want.abs().amax((0, 1)) > most / 2    # (past fp16: its infinity)
    assert over.sum() < D // 2
    check(out.masked_fill(over, 0), q, k, v.masked_fill(over, 0), lens, floor)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_values_at_the_limit_that_a_row_does_not_see(tq, dtype, call):  # noqa: F811
    """A block whose scale is the largest: values of 2^128, past what bf16 holds, at later positions and any bytes behind
    the end must not reach the rows before them."""
    gen = torch.Generator().manual_seed(63)
    n = 180
    s = Setup(tq, gen, [n], 1, 16)
    K, V = (torch.randn(n, 1, D, generator=gen).bfloat16() for _ in range(2))
    V[100, 0, ::7] = torch.finfo(torch.bfloat16).max     # its block's values get the scale 2^120, itself the code of 256
    p, sc = R.write(s.pool.cpu(), s.scales.cpu(), K, V, [0, n], [0], s.rows)
    s.pool.copy_(p)
    s.scales.copy_(sc)
    assert float(s.scales[s.rows[0][100 // 16], 0, 1]) == 2.0 ** 120
    q = torch.randn(n, 4, D, generator=gen).to(DT[dtype]).cuda()
    k, v = R.stored(s.pool, s.scales, s.rows[0], n)
    if call == "decode":
        out = s.cache.decode(q[:100], s.table.repeat(100, 1), i32(list(range(1, 101))))
    else:
        out = s.cache.prefill(q, i32([0, n]), i32([0]), s.table)[:100]
    check(out, q[:100], k, v, list(range(1, 101)), DECODE if call == "decode" else PREFILL)


@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_any_bytes_behind_the_end_of_a_block_of_the_largest_scale(tq, call):  # noqa: F811
    gen = torch.Generator().manual_seed(64)
    n = 37
    s = Setup(tq, gen, [n], 1, 16)
    s.fill([n])
    blk = s.rows[0][2]
    s.scales[blk, 0, 1] = 2.0 ** 120
    s.pool[blk, 0, 1, :5] &= 0x87                          # live values of 2^111 .. 2^114
    s.pool[blk, 0, 1, 5:] = torch.randint(0x78, 0x80, (11, D), generator=gen).to(torch.uint8).cuda()
    q = torch.randn(5, 4, D, generator=gen).bfloat16().cuda()
    k, v = R.stored(s.pool, s.scales, s.rows[0], n)
    if call == "decode":
        out = s.cache.decode(q, s.table.repeat(5, 1), i32([33, 34, 35, 36, 37]))
    else:
        out = s.cache.prefill(q, i32([0, 5]), i32([32]), s.table)
    check(out, q, k, v, [33, 34, 35, 36, 37], DECODE if call == "decode" else PREFILL)
