"""The 8-bit paged cache on the GPU: codes of NaN, values at the ends of the range, and slots that a row does not see."""
import math

import pytest
import torch

from tests import fp8_reference as R
from tests.test_gpu_fp8 import D, DECODE, DT, PREFILL, Setup, check, i32, tq  # noqa: F401

pytestmark = pytest.mark.gpu


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
