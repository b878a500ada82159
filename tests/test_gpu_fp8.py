"""The 8-bit paged cache on the GPU: write, read back, one-token and chunk
attention, each against its float64 form, and the four run together."""
import math

import pytest
import torch

from tests import fp8_reference as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
D = 128


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from online_kv_cache_encode_gb300 import build
    build.build()
    from online_kv_cache_encode_gb300 import tq as T
    return T


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Setup:
    """A pool of random bytes (so also NaN codes) and garbage scales, and a batch's blocks anywhere in it."""

    def __init__(self, tq, gen, lens, hkv, bs, spare=3):
        need = [-(-n // bs) for n in lens]
        nb = max(1, sum(need)) + spare
        self.gen, self.hkv, self.bs, self.nb = gen, hkv, bs, nb
        self.pool = torch.randint(0, 256, (nb, hkv, 2, bs, D), dtype=torch.uint8, generator=gen).cuda()
        self.scales = torch.full((nb, hkv, 2), math.nan).cuda()
        order = torch.randperm(nb, generator=gen).tolist()
        mb = max(1, max(need)) + 1
        self.rows, at = [], 0
        for n in need:
            self.rows.append(order[at:at + n] + [-1] * (mb - n))
            at += n
        self.table = i32(self.rows)
        self.free = order[at:]
        self.cache = tq.Fp8Cache(nb, hkv, block_size=bs, pool=self.pool.view(-1), scales=self.scales)

    def fill(self, lens, outliers=True):
        """Every sequence's first lens[b] positions, written by the reference."""
        T = sum(lens)
        K, V = (torch.randn(T, self.hkv, D, generator=self.gen) for _ in range(2))
        if outliers:
            K[..., 5] *= 20
            V *= torch.exp(torch.randn(T, 1, 1, generator=self.gen))
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        p, s = R.write(self.pool.cpu(), self.scales.cpu(), K, V, cu, [0] * len(lens), self.rows)
        self.pool.copy_(p)
        self.scales.copy_(s)


def cu_of(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


# --------------------------------------------------------------------------- write
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("hkv,starts,news", [
    (1, [0], [1]),
    (2, [0, 5, 130, 16], [3, 0, 40, 16]),
    (3, [15, 127, 0, 64, 129], [1, 2, 257, 1, 128]),
    (8, [7] * 40, [1] * 40),
])
def test_write_bytes(tq, dtype, bs, hkv, starts, news):
    """Every byte of the pool and every scale: new codes, codes moved to a larger scale, the rest untouched."""
    gen = torch.Generator().manual_seed(bs * 1000 + hkv)
    s = Setup(tq, gen, [a + n for a, n in zip(starts, news)], hkv, bs)
    s.fill(starts)
    T, pad = sum(news), 3
    big = torch.randn(T + pad, hkv, 2, 1, generator=gen).mul(2).exp()  # rows of very different size
    kv = (torch.randn(T + pad, hkv, 2, D, generator=gen) * big).to(DT[dtype])
    cu = cu_of(news)
    want, wants = R.write(s.pool.cpu(), s.scales.cpu(), kv[:, :, 0], kv[:, :, 1], cu, starts, s.rows)
    st = tq.new_status()
    kv = kv.cuda()
    s.cache.write(kv[:, :, 0], kv[:, :, 1], i32(cu), i32(starts), s.table, status=st)
    assert st.item() == 0
    live = ~torch.isnan(wants)
    assert torch.equal(s.scales.cpu()[live], wants[live])
    assert torch.isnan(s.scales.cpu()[~live]).all()
    assert torch.equal(s.pool.cpu(), want)


def test_write_token_by_token(tq):
    """Appends that raise a block's scale step by step, and appends that do not, as the reference does them."""
    gen = torch.Generator().manual_seed(3)
    s = Setup(tq, gen, [70], 2, 32)
    p, sc = s.pool.cpu(), s.scales.cpu()
    for t in range(70):
        kv = torch.randn(1, 4, D, generator=gen).mul(2.0 ** (t % 9)).bfloat16()
        p, sc = R.write(p, sc, kv[:, :2], kv[:, 2:], [0, 1], [t], s.rows)
        kv = kv.cuda()
        s.cache.write(kv[:, :2], kv[:, 2:], i32([0, 1]), i32([t]), s.table)
    live = ~torch.isnan(sc)
    assert torch.equal(s.pool.cpu(), p) and torch.equal(s.scales.cpu()[live], sc[live])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_write_extremes(tq, dtype):
    """Zeros, the type's largest and smallest values, exact borders of the scale, infinities and NaN."""
    t = DT[dtype]
    fi = torch.finfo(t)
    gen = torch.Generator().manual_seed(9)
    s = Setup(tq, gen, [16] * 6, 1, 16)
    K = torch.zeros(96, 1, D, dtype=t)
    K[16:32] = fi.max
    K[32:48, :, ::3] = fi.tiny
    K[48:64] = 448.0
    K[49, 0, 1] = -448.0 * (1 + fi.eps)     # one step above: the next scale
    K[64:80] = torch.randn(16, 1, D, generator=gen).to(t)
    K[80:96] = torch.randn(16, 1, D, generator=gen).to(t)
    V = K.flip(2).clone()
    K[70, 0, 3], K[71, 0, 4], K[72, 0, 5] = math.inf, -math.inf, math.nan
    V[80:96] = math.nan
    cu = cu_of([16] * 6)
    want, wants = R.write(s.pool.cpu(), s.scales.cpu(), K, V, cu, [0] * 6, s.rows)
    st = tq.new_status()
    s.cache.write(K.cuda(), V.cuda(), i32(cu), i32([0] * 6), s.table, status=st)
    assert st.item() == tq.FLAG_NONFINITE
    live = ~torch.isnan(wants)
    assert torch.equal(s.scales.cpu()[live], wants[live])
    assert torch.equal(s.pool.cpu(), want)


def test_bad_blocks_and_starts(tq):
    """Ids outside the pool, positions past the table and negative starts are flagged and skipped, by every call."""
    gen = torch.Generator().manual_seed(4)
    s = Setup(tq, gen, [64, 64, 64], 2, 16)
    s.fill([64, 64, 64])
    rows = [list(r) for r in s.rows]
    rows[0][1], rows[1][0] = s.nb, -7        # second block of 0, first of 1
    table = i32(rows)
    before, sbefore = s.pool.clone(), s.scales.clone()
    K = torch.randn(40 + 40 + 8 + 5, 2, D, generator=gen).bfloat16().cuda()
    # sequence 2: position 80 .. 87 lies past the five blocks of the table
    args = (i32([0, 40, 80, 88]), i32([0, -3, 80]), table)
    st = tq.new_status()
    s.cache.write(K, K, *args, status=st)
    assert st.item() == tq.FLAG_BAD_SLOT
    want, wants = R.write(before.cpu(), sbefore.cpu(), K[:16].cpu(), K[:16].cpu(), [0, 16], [0], s.rows[:1])
    want, wants = R.write(want, wants, K[32:40].cpu(), K[32:40].cpu(), [0, 8], [32], s.rows[:1])
    assert torch.equal(s.pool.cpu(), want)
    out = tuple(torch.full((93, 2, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = tq.new_status()
    s.cache.read(*args, 93, torch.bfloat16, out=out, status=st)
    assert st.item() == tq.FLAG_BAD_SLOT
    for o in out:
        assert (o[16:32] == 7).all() and (o[40:] == 7).all() and not (o[:16] == 7).all()
    q = torch.randn(93, 4, D, generator=gen).bfloat16().cuda()
    o = torch.full((93, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    st = tq.new_status()
    s.cache.prefill(q, *args, out=o, status=st)
    assert st.item() == tq.FLAG_BAD_SLOT
    assert (o[88:] == 7).all()
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[16:32] = False
    row = [r if 0 <= r < s.nb else 0 for r in rows[0]]
    check(o[:40], q[:40], *R.stored(s.pool, s.scales, row, 40), [i + 1 for i in range(40)], PREFILL, keep=keep)
    lens = i32([-5, 1000, 16])
    st = tq.new_status()
    o = s.cache.decode(q[:3], table, lens, status=st)
    assert st.item() == tq.FLAG_BAD_SLOT and (o[0] == 0).all()
    check(o[2:], q[2:3], *R.stored(s.pool, s.scales, rows[2], 16), [16], DECODE)


# --------------------------------------------------------------------------- read
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_read_back(tq, dtype, bs):
    gen = torch.Generator().manual_seed(bs)
    lens, starts, news = [300, 0, 129, 128, 64, 1], [37, 0, 128, 0, 63, 0], [263, 0, 1, 128, 1, 1]
    s = Setup(tq, gen, lens, 3, bs)
    s.fill(lens)
    T = sum(news)
    out = tuple(torch.full((T + 4, 3, D), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    st = tq.new_status()
    s.cache.read(i32(cu_of(news)), i32(starts), s.table, T + 4, DT[dtype], out=out, status=st)
    assert st.item() == 0
    at = 0
    for b, (a, n) in enumerate(zip(starts, news)):
        if n:
            for got, want in zip(out, R.stored(s.pool, s.scales, s.rows[b], a + n)):
                assert torch.equal(got[at:at + n], want[:, a:].permute(1, 0, 2).to(DT[dtype]))
        at += n
    assert all((o[T:] == 7).all() for o in out)
    fresh = s.cache.read(i32(cu_of(news)), i32(starts), s.table, T, DT[dtype])
    assert all(torch.equal(f, o[:T]) for f, o in zip(fresh, out))


# --------------------------------------------------------------------------- attention
# An element of a query far below its row's largest one is held in steps of that one's size: three terms 1/16 apart
# reach below 2^-21 of it (decode), terms that share one accumulator end at half a step of 2^-9 against at least 224,
# 2^-17.8 (prefill); as multiples of 2^-16:
DECODE, PREFILL = 2.0 ** -5, 2.0 ** -1.8


def check(out, q, k, v, limits, floor, sm_scale=1 / math.sqrt(D), keep=None):
    """|out - exact| within what the roundings allow, element by element:
      the output's own rounding       eps / 2 |out|
      each weight rounded to 2 (bf16) or 3 (fp16) terms of 4 bits, or to bf16 and to two terms of bf16:
                                      at most 2^-8 and 2^-12 of it, so that much of sum w |v|
      a score's 128 products and their sums in fp32, u = 2^-23 each (truncated), and its share in numerator
      and denominator                 2 * 2^-16 * max_t sum |q k_t| sm_scale of sum w |v|
      exponentials, sums over tokens and joins in fp32, about 2^-19 of sum w |v|."""
    want, spread, sharp = R.attend(q, k, v, limits, sm_scale, keep, floor)
    eps = torch.finfo(out.dtype).eps
    weights = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -12
    tol = eps / 2 * want.abs() + spread * (weights + 2.0 ** -19 + 2 * 2.0 ** -16 * sharp[..., None])
    tol = tol + (2.0 ** -25 if out.dtype == torch.float16 else 0)  # fp16 subnormals
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv,lens", [
    (1, 1, [1]),
    (8, 1, [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 0]),
    (20, 20, [700, 0, 33]),
    (15, 3, [1000, 1]),
    (32, 2, [513, 64, 640]),
    (40, 2, [300, 77]),
    (128, 1, [200]),
])
def test_decode(tq, dtype, bs, hq, hkv, lens):
    gen = torch.Generator().manual_seed(hq * 100 + bs)
    s = Setup(tq, gen, lens, hkv, bs)
    s.fill(lens)
    wide = torch.randn(len(lens), hq + 3, D, generator=gen).to(DT[dtype]).cuda()
    q = wide[:, 2:2 + hq]
    st = tq.new_status()
    out = s.cache.decode(q, s.table, i32(lens), status=st)
    assert st.item() == 0
    for b, n in enumerate(lens):
        k, v = R.stored(s.pool, s.scales, s.rows[b], n)
        check(out[b:b + 1], q[b:b + 1], k, v, [n], DECODE)
        if n == 0:
            assert (out[b] == 0).all()
    again = s.cache.decode(q, s.table, i32(lens))
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bs,hq,hkv,starts,news", [
    (16, 1, 1, [0], [1]),
    (16, 8, 1, [0, 100, 5, 0], [130, 17, 0, 1]),
    (32, 6, 2, [127, 128, 0], [2, 300, 129]),
    (64, 20, 20, [333, 1], [70, 200]),
    (128, 32, 2, [500], [33]),
    (16, 40, 1, [0, 900], [64, 9]),
    (16, 128, 1, [250], [5]),
    (32, 7, 1, [63, 0], [40, 128]),
])
def test_prefill(tq, dtype, bs, hq, hkv, starts, news):
    gen = torch.Generator().manual_seed(hq * 10 + bs)
    lens = [a + n for a, n in zip(starts, news)]
    s = Setup(tq, gen, lens, hkv, bs)
    s.fill(lens)
    T = sum(news)
    q = torch.randn(T + 2, hq + 2, D, generator=gen).to(DT[dtype]).cuda()[:, 1:1 + hq]
    out = torch.full((T + 2, hq, D), 7.0, dtype=DT[dtype], device="cuda")
    st = tq.new_status()
    s.cache.prefill(q, i32(cu_of(news)), i32(starts), s.table, out=out, status=st)
    assert st.item() == 0 and (out[T:] == 7).all()
    at = 0
    for b, (a, n) in enumerate(zip(starts, news)):
        if n:
            k, v = R.stored(s.pool, s.scales, s.rows[b], a + n)
            check(out[at:at + n], q[at:at + n], k, v, [a + i + 1 for i in range(n)], PREFILL)
        at += n


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,batch", [(16, 8, 24), (16, 8, 33), (32, 2, 24), (20, 20, 2)])
def test_prefill_of_many_units(tq, dtype, hq, hkv, batch):
    """More units than SMs, of all lengths and equal ones: sequences without new tokens, with one, behind long prefixes,
    one with a negative start (flagged, its rows are zero), rows behind the last sequence, padding's empty sequences."""
    gen = torch.Generator().manual_seed(53)
    starts = torch.randint(0, 500, (batch,), generator=gen).tolist()
    news = torch.randint(0, 1 + 3000 // batch, (batch,), generator=gen).tolist()
    starts[0], news[0] = 0, 1500 // batch * 2
    if batch > 2:
        starts[1], news[1] = 700, 1
        starts[2], news[2] = 40, 0
        starts[3:6], news[3:6] = [128] * 3, [130] * 3
        starts[6], news[6] = -9, 50
        news[-1] = 0
    lens = [max(a, 0) + n for a, n in zip(starts, news)]
    s = Setup(tq, gen, lens, hkv, 64)
    s.fill(lens)
    T = sum(news)
    q = torch.randn(T + 5, hq, D, generator=gen).to(DT[dtype]).cuda()
    out, st = torch.full_like(q, 7), tq.new_status()
    s.cache.prefill(q, i32(cu_of(news)), i32(starts), s.table, out=out, status=st)
    assert st.item() == (tq.FLAG_BAD_SLOT if batch > 2 else 0)
    assert (out[T:] == 7).all()
    at = 0
    for b, (a, n) in enumerate(zip(starts, news)):
        if n and a < 0:
            assert not out[at:at + n].any()
        elif n:
            k, v = R.stored(s.pool, s.scales, s.rows[b], a + n)
            check(out[at:at + n], q[at:at + n], k, v, [a + i + 1 for i in range(n)], PREFILL)
        at += n


def sink_case(tq, dtype, call, gen):
    """One token that takes nearly all of the weight and 4000 others that matter together, with blocks of values of
    very different size: small weights and small scales keep their precision."""
    n = 4000
    s = Setup(tq, gen, [n], 1, 16)
    K, V = (torch.randn(n, 1, D, generator=gen) for _ in range(2))
    q = torch.randn(1, 8, D, generator=gen).to(DT[dtype])
    K[0, 0] = q[0].float().mean(0) * 60
    V[0] = 2.0 ** -10
    V *= torch.pow(2.0, torch.randint(-6, 7, (n // 16, 1, 1), generator=gen).float()).repeat_interleave(16, 0)
    p, sc = R.write(s.pool.cpu(), s.scales.cpu(), K, V, [0, n], [0], s.rows)
    s.pool.copy_(p)
    s.scales.copy_(sc)
    q = q.cuda()
    out = s.cache.decode(q, s.table, i32([n])) if call == "decode" else s.cache.prefill(q, i32([0, 1]), i32([n - 1]), s.table)
    check(out, q, *R.stored(s.pool, s.scales, s.rows[0], n), [n], DECODE if call == "decode" else PREFILL)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_one_token_takes_most_weight(tq, dtype, call):
    sink_case(tq, dtype, call, torch.Generator().manual_seed(77))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("step", [3.0, 40.0, -40.0])
def test_scores_that_rise_and_fall(tq, dtype, step):
    """Scores whose size changes by many octaves from tile to tile, up and down: every reference has to follow."""
    gen = torch.Generator().manual_seed(21)
    n = 1100
    s = Setup(tq, gen, [n], 1, 16)
    q = torch.randn(300, 2, D, generator=gen).to(DT[dtype])
    q[:, 1] = -q[:, 0]                       # one head's rising scores are the other's falling ones
    q[1:] = q[:1] * (1 + 0.01 * torch.randn(299, 1, 1, generator=gen)).to(DT[dtype])
    unit = q[0, 0].float() / q[0, 0].float().norm()
    K, V = (torch.randn(n, 1, D, generator=gen) for _ in range(2))
    K[:, 0] += unit * step * torch.arange(n)[:, None] / 64
    p, sc = R.write(s.pool.cpu(), s.scales.cpu(), K, V, [0, n], [0], s.rows)
    s.pool.copy_(p)
    s.scales.copy_(sc)
    q = q.cuda()
    k, v = R.stored(s.pool, s.scales, s.rows[0], n)
    out = s.cache.prefill(q, i32([0, 300]), i32([n - 300]), s.table)
    check(out, q, k, v, [n - 300 + i + 1 for i in range(300)], PREFILL)
    for m in (n, 700, 257):
        check(s.cache.decode(q[:1], s.table, i32([m])), q[:1], k[:, :m], v[:, :m], [m], DECODE)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("call", ["decode", "prefill"])
@pytest.mark.parametrize("octaves", [7, 20, 60, 165])
def test_large_values_of_negligible_weight(tq, dtype, call, octaves):
    """Blocks whose values are 2^octaves the others' size but whose weights are 2^-(octaves + 20) and less: they must
    not cost the others' weights their bits.  In some tiles only, and with a head for which the same blocks weigh in."""
    gen = torch.Generator().manual_seed(31)
    n = 900
    s = Setup(tq, gen, [n], 1, 16)
    K, V = (torch.randn(n, 1, D, generator=gen) for _ in range(2))
    q = torch.randn(1, 3, D, generator=gen).to(DT[dtype])
    u = q[0, 0].float()
    q[0, 1] = -q[0, 0] / 64
    big = torch.zeros(n, dtype=torch.bool)
    big[32:48] = big[256 + 80:256 + 112] = big[896:] = True
    K[big, 0] -= u * (octaves + 40) * math.log(2) * math.sqrt(D) / float(u @ u)
    if octaves > 100:
        V *= 2.0 ** -85
    V[big] *= 2.0 ** octaves
    V[512:528] = 0                               # a block of zeros has the least scale
    p, sc = R.write(s.pool.cpu(), s.scales.cpu(), K, V, [0, n], [0], s.rows)
    s.pool.copy_(p)
    s.scales.copy_(sc)
    q = q.cuda()
    out = s.cache.decode(q, s.table, i32([n])) if call == "decode" else s.cache.prefill(q, i32([0, 1]), i32([n - 1]), s.table)
    k, v = R.stored(s.pool, s.scales, s.rows[0], n)
    floor, most = DECODE if call == "decode" else PREFILL, torch.finfo(out.dtype).max
    want = R.attend(q, k, v, [n], 1 / math.sqrt(D), None, floor)[0]
    fits = [h for h in range(3) if want[0, h].abs().max() < most / 2]
    assert 0 in fits
    check(out[:, fits], q[:, fits], k, v, [n], floor)
    over = want.abs() > 2 * most                 # (past fp16: its infinity)
    assert torch.equal(out[over].double(), want[over].sign() * math.inf)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bs", [16, 64])
def test_runs_of_tiles_with_and_without_far_scales(tq, dtype, bs):
    """The same blocks read by 300 sequences of other lengths, so that a CTA goes through several tiles whose value
    scales lie far apart in some and near in others, and through several sequences."""
    gen = torch.Generator().manual_seed(37)
    n, B = 1500, 300
    s = Setup(tq, gen, [n], 1, bs)
    K, V = (torch.randn(n, 1, D, generator=gen) for _ in range(2))
    u = torch.randn(D, generator=gen)
    q = (u * (1 + 0.05 * torch.randn(B, 10, 1, generator=gen))).to(DT[dtype])
    q[::2, 1:3] = (torch.randn((B + 1) // 2, 2, D, generator=gen)).to(DT[dtype])
    big = torch.zeros(n, dtype=torch.bool)
    big[64:128] = big[832:896] = big[1472:] = True
    K[big, 0] -= u * 40 * math.log(2) * math.sqrt(D) / float(u @ u)
    V[big] *= 2.0 ** 10
    V[320:384] *= 2.0 ** -12
    p, sc = R.write(s.pool.cpu(), s.scales.cpu(), K, V, [0, n], [0], s.rows)
    s.pool.copy_(p)
    s.scales.copy_(sc)
    lens = torch.randint(0, n + 1, (B,), generator=gen).tolist()
    lens[:4] = [0, 1, n, n]
    q = q.cuda()
    k, v = R.stored(s.pool, s.scales, s.rows[0], n)
    table = s.table.repeat(B, 1)
    for heads in (3, 10):
        out = s.cache.decode(q[:, :heads], table, i32(lens))
        assert not out[0].any()
        check(out[1:], q[1:, :heads], k, v, lens[1:], DECODE)


@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_large_and_small_scales(tq, call):
    """Blocks of zeros, of values near the type's limits and of tiny ones, in one sequence; queries of any size."""
    gen = torch.Generator().manual_seed(5)
    n = 300
    s = Setup(tq, gen, [n], 1, 16)
    K, V = (torch.randn(n, 1, D, generator=gen).bfloat16() for _ in range(2))
    V[0:16], V[16:32], V[32:48] = 0, V[16:32] * 2.0 ** 100, V[32:48] * 2.0 ** -100
    K[48:64], K[64:80] = 0, K[64:80] * 2.0 ** -90
    p, sc = R.write(s.pool.cpu(), s.scales.cpu(), K, V, [0, n], [0], s.rows)
    s.pool.copy_(p)
    s.scales.copy_(sc)
    q = torch.randn(1, 4, D, generator=gen).bfloat16()
    q[0, 1] *= 2.0 ** -80
    q[0, 2] = 0
    q[0, 3] *= 8
    q = q.cuda()
    out = s.cache.decode(q, s.table, i32([n])) if call == "decode" else s.cache.prefill(q, i32([0, 1]), i32([n - 1]), s.table)
    check(out, q, *R.stored(s.pool, s.scales, s.rows[0], n), [n], DECODE if call == "decode" else PREFILL)


def test_binding_refusals(tq):
    """What the binding and the library refuse, with nothing launched."""
    s = Setup(tq, torch.Generator().manual_seed(1), [40], 2, 16)
    c, cu, st, ln = s.cache, i32([0, 4]), i32([0]), i32([4])
    K = torch.zeros(4, 2, D, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 4, D, dtype=torch.bfloat16, device="cuda")
    before = s.pool.clone()
    for call in (lambda: c.write(K[:, :1], K[:, :1], cu, st, s.table), lambda: c.write(K, K[:3], cu, st, s.table),
                 lambda: c.write(K, K.half(), cu, st, s.table), lambda: c.write(K, K, cu.long(), st, s.table),
                 lambda: c.write(K, K, cu[:1], st, s.table), lambda: c.write(K.cpu(), K.cpu(), cu, st, s.table),
                 lambda: c.write(K, K, cu, st.cpu(), s.table), lambda: c.write(K, K, cu, st, s.table.t()),
                 lambda: c.write(K[..., ::2], K[..., ::2], cu, st, s.table),
                 lambda: c.decode(q, s.table, ln.long()), lambda: c.decode(q, s.table.long(), ln),
                 lambda: c.decode(q[..., :64], s.table, ln), lambda: c.decode(q, s.table, i32([1, 2])),
                 lambda: c.decode(q, s.table, ln, out=q.half()), lambda: c.decode(q, s.table, ln, out=q.expand(1, 4, D)[:, :2]),
                 lambda: c.decode(q, s.table, ln, workspace=torch.zeros(1 << 24, dtype=torch.uint8)),
                 lambda: c.prefill(q, i32([0, 1]), st, s.table, workspace=torch.zeros(1 << 24, dtype=torch.uint8)),
                 lambda: c.read(cu, st, s.table, 4, torch.bfloat16, out=(K, K.half())),
                 lambda: c.prefill(q, cu, st, s.table, status=torch.zeros(1, device="cuda"))):
        with pytest.raises(AssertionError):
            call()
    for call, status in ((lambda: c.decode(q.float(), s.table, ln), tq.TQ_ERR_UNSUPPORTED),
                         (lambda: c.prefill(q.float(), i32([0, 1]), st, s.table), tq.TQ_ERR_UNSUPPORTED),
                         (lambda: c.decode(q[:, :3], s.table, ln), tq.TQ_ERR_INVALID_ARG),
                         (lambda: c.decode(q, s.table, ln, sm_scale=-1.0), tq.TQ_ERR_INVALID_ARG),
                         (lambda: c.decode(q, s.table, ln, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")),
                          tq.TQ_ERR_WORKSPACE),
                         (lambda: c.write(K.view(-1)[4:4 + 3 * 2 * D].view(3, 2, D), K[:3], cu, st, s.table),
                          tq.TQ_ERR_INVALID_ARG)):
        with pytest.raises(tq.TQError) as e:
            call()
        assert e.value.status == status
    torch.cuda.synchronize()
    assert torch.equal(s.pool, before)
    # nothing to do is not an error
    none = K[:0]
    c.write(none, none, i32([0, 0]), st, s.table)
    assert c.decode(q[:0], s.table[:0], ln[:0]).shape == (0, 4, D)
    assert c.prefill(q[:0], i32([0, 0]), st, s.table).shape == (0, 4, D)
    assert c.read(i32([0, 0]), st, s.table, 0)[0].shape == (0, 2, D)


@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_nonfinite_query_stays_in_its_row(tq, call):
    gen = torch.Generator().manual_seed(6)
    s = Setup(tq, gen, [200], 1, 16)
    s.fill([200])
    q = torch.randn(1, 8, D, generator=gen).bfloat16().cuda()
    bad = q.clone()
    bad[0, 2, 7], bad[0, 5, 9] = math.nan, math.inf
    run = (lambda x: s.cache.decode(x, s.table, i32([200]))) if call == "decode" else (
        lambda x: s.cache.prefill(x, i32([0, 1]), i32([199]), s.table))
    good, out = run(q), run(bad)
    rest = [0, 1, 3, 4, 6, 7]
    assert torch.equal(out[0, rest], good[0, rest])
    assert torch.isnan(out[0, [2, 5]]).all()


# --------------------------------------------------------------------------- together
def test_serving_run(tq):
    """Two prompts written in chunks with attention over each chunk, then steps of one token each, then read back."""
    gen = torch.Generator().manual_seed(8)
    lens, hkv, hq = [150, 37], 2, 8
    total = [n + 5 for n in lens]
    s = Setup(tq, gen, total, hkv, 16)
    pool, scales = s.pool.cpu(), s.scales.cpu()
    qkv = [torch.randn(n, hq + 2 * hkv, D, generator=gen).bfloat16() for n in total]
    done = [0, 0]
    for news in ([64, 37], [86, 0], [1, 1], [1, 1], [1, 1], [1, 1], [1, 1]):
        rows = torch.cat([qkv[b][done[b]:done[b] + n] for b, n in enumerate(news)]).cuda()
        q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        cu, start = cu_of(news), list(done)
        pool, scales = R.write(pool, scales, k.cpu(), v.cpu(), cu, start, s.rows)
        s.cache.write(k, v, i32(cu), i32(start), s.table)
        if news == [1, 1]:
            out = s.cache.decode(q, s.table, i32([a + 1 for a in start]))
        else:
            out = s.cache.prefill(q, i32(cu), i32(start), s.table)
        assert torch.equal(s.pool.cpu(), pool)
        for b, n in enumerate(news):
            if n:
                kk, vv = R.stored(s.pool, s.scales, s.rows[b], start[b] + n)
                check(out[cu[b]:cu[b + 1]], q[cu[b]:cu[b + 1]], kk, vv, [start[b] + i + 1 for i in range(n)],
                      DECODE if news == [1, 1] else PREFILL)
            done[b] += n
    K, V = s.cache.read(i32(cu_of(total)), i32([0, 0]), s.table, sum(total), torch.float32)
    for b, n in enumerate(total):
        kk, vv = R.stored(s.pool, s.scales, s.rows[b], n)
        at = cu_of(total)[b]
        assert torch.equal(K[at:at + n].double(), kk.permute(1, 0, 2)) and torch.equal(V[at:at + n].double(), vv.permute(1, 0, 2))


def test_captured_steps(tq):
    """A write and a decode captured once and replayed as the sequences grow; eager calls between the replays."""
    gen = torch.Generator().manual_seed(10)
    hkv, hq, B = 2, 16, 3
    lens = [120, 5, 300]
    s = Setup(tq, gen, [n + 6 for n in lens], hkv, 16)
    s.fill(lens)
    x = torch.zeros(B, hq + 2 * hkv, D, dtype=torch.bfloat16, device="cuda")
    cu, start, ln = i32([0, 1, 2, 3]), i32(lens), i32([n + 1 for n in lens])
    step = lambda: (s.cache.write(x[:, hq:hq + hkv], x[:, hq + hkv:], cu, start, s.table),  # noqa: E731
                    s.cache.decode(x[:, :hq], s.table, ln))[1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = s.pool.clone(), s.scales.clone()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    s.pool.copy_(keep[0])
    s.scales.copy_(keep[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t in range(6):
        x.copy_(torch.randn(x.shape, generator=gen).bfloat16())
        graph.replay()
        n = [a + t + 1 for a in lens]
        eager = s.cache.decode(x[:, :hq], s.table, i32(n))
        assert torch.equal(out, eager)
        for b in range(B):
            check(out[b:b + 1], x[b:b + 1, :hq], *R.stored(s.pool, s.scales, s.rows[b], n[b]), [n[b]], DECODE)
        start += 1
        ln += 1


def test_captured_prompt(tq):
    """A chunk's write, its attention (split over the tokens, so with a workspace) and a read back, captured once and
    replayed with other rows, positions and lengths, an idle sequence and rows behind the last one among them."""
    gen = torch.Generator().manual_seed(41)
    lens, hq, hkv, T = [900, 300], 4, 2, 96
    s = Setup(tq, gen, lens, hkv, 32)
    K, V = (torch.randn(T, hkv, D, generator=gen).bfloat16().cuda() for _ in range(2))
    q = torch.randn(T, hq, D, generator=gen).bfloat16().cuda()
    cu, st = i32([0, 0, 0]), i32([0, 0])
    cu_all, zero = i32([0, 900, 1200]), i32([0, 0])
    prefix = [torch.randn(1200, hkv, D, generator=gen).bfloat16().cuda() for _ in range(2)]
    out, back = torch.empty_like(q), (torch.empty_like(K), torch.empty_like(V))

    def step():
        s.cache.write(K, V, cu, st, s.table)
        s.cache.prefill(q, cu, st, s.table, out=out)
        s.cache.read(cu, st, s.table, T, out=back)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for cut, start in (([0, 96, 96], [800, 0]), ([0, 40, 90], [13, 250]), ([0, 0, 1], [5, 299]), ([0, 50, 96], [0, 0])):
        s.cache.write(*prefix, cu_all, zero, s.table)
        K.copy_(torch.randn(T, hkv, D, generator=gen))
        V.copy_(torch.randn(T, hkv, D, generator=gen))
        q.copy_(torch.randn(T, hq, D, generator=gen))
        cu.copy_(i32(cut))
        st.copy_(i32(start))
        for x in (out, *back):
            x.fill_(7)
        want = [x.cpu() for x in (s.pool, s.scales)]
        graph.replay()
        want = R.write(*want, K.cpu().float(), V.cpu().float(), cut, start, s.rows)
        assert torch.equal(s.pool.cpu(), want[0])
        assert torch.equal(s.scales.cpu().view(torch.int32), want[1].view(torch.int32))
        for b in range(2):
            a, z = cut[b], cut[b + 1]
            if z > a:
                k, v = R.stored(s.pool, s.scales, s.rows[b], start[b] + z - a)
                check(out[a:z], q[a:z], k, v, [start[b] + i + 1 for i in range(z - a)], PREFILL)
                for x, y in zip(back, (k, v)):
                    assert torch.equal(x[a:z], y[:, start[b]:].permute(1, 0, 2).to(torch.bfloat16))
        for x in (out, *back):
            assert (x[cut[-1]:] == 7).all()


def test_one_workspace_for_calls_of_all_shapes(tq):
    """Small and large batches and head counts in turn on the cache's kept workspace, whose counters must be found at
    zero by each, and on one that the caller passes."""
    gen = torch.Generator().manual_seed(14)
    lens = [1500] + [300] * 40
    s = Setup(tq, gen, lens, 4, 16)
    s.fill(lens, outliers=False)
    q = torch.randn(41, 64, D, generator=gen).bfloat16().cuda()
    own = torch.zeros(s.cache._lib.tq_fp8_decode_workspace_bytes(s.cache._h, 41, 64), dtype=torch.uint8, device="cuda")
    cases = [(1, 4), (41, 64), (1, 64), (20, 4), (41, 32), (2, 8), (41, 64), (1, 4)]
    fresh = []
    for B, hq in cases:
        ws = torch.zeros_like(own)
        fresh.append(s.cache.decode(q[:B, :hq], s.table[:B], i32(lens[:B]), workspace=ws))
    for _ in range(3):
        for (B, hq), want in zip(cases, fresh):
            assert torch.equal(s.cache.decode(q[:B, :hq], s.table[:B], i32(lens[:B])), want)
            assert torch.equal(s.cache.decode(q[:B, :hq], s.table[:B], i32(lens[:B]), workspace=own), want)


def test_two_streams_at_once(tq):
    """Decodes and prefills of the same cache issued on two streams without waiting for one another."""
    gen = torch.Generator().manual_seed(11)
    lens = [3000, 1700]
    s = Setup(tq, gen, lens, 1, 16)
    s.fill(lens)
    q = torch.randn(2, 8, D, generator=gen).bfloat16().cuda()
    q2 = torch.randn(40, 8, D, generator=gen).bfloat16().cuda()
    one, chunk = i32(lens), (i32([0, 20, 40]), i32([n - 20 for n in lens]))
    want, want2 = s.cache.decode(q, s.table, one), s.cache.prefill(q2, *chunk, s.table)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(20):
        for st in streams:
            with torch.cuda.stream(st):
                got.append((s.cache.decode(q, s.table, one), s.cache.prefill(q2, *chunk, s.table)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, want2) for a, b in got)


def test_pool_beyond_32_bits(tq):
    """Blocks whose codes lie past 4 GB of the pool."""
    gen = torch.Generator().manual_seed(12)
    hkv, bs = 8, 128
    nb = (9 << 29) // (hkv * 2 * bs * D)   # 4.5 GB
    pool = torch.zeros(nb * hkv * 2 * bs * D, dtype=torch.uint8, device="cuda")
    scales = torch.ones(nb, hkv, 2, device="cuda")
    c = tq.Fp8Cache(nb, hkv, block_size=bs, pool=pool, scales=scales)
    rows = [[nb - 1, 3, nb - 2]]
    K, V = (torch.randn(300, hkv, D, generator=gen).bfloat16() for _ in range(2))
    c.write(K.cuda(), V.cuda(), i32([0, 300]), i32([0]), i32(rows))
    small = torch.zeros(3, hkv, 2, bs, D, dtype=torch.uint8)
    want, wants = R.write(small, torch.ones(3, hkv, 2), K, V, [0, 300], [0], [[2, 0, 1]])
    view = pool.view(nb, hkv, 2, bs, D)
    assert torch.equal(view[[3, nb - 2, nb - 1]].cpu(), want) and torch.equal(scales[[3, nb - 2, nb - 1]].cpu(), wants)
    k, v = R.stored(want.cuda(), wants.cuda(), [2, 0, 1], 300)
    q = torch.randn(3, 16, D, generator=gen).bfloat16().cuda()
    check(c.decode(q[:1], i32(rows), i32([300])), q[:1], k, v, [300], DECODE)
    check(c.prefill(q, i32([0, 3]), i32([297]), i32(rows)), q, k, v, [298, 299, 300], PREFILL)
    got = c.read(i32([0, 300]), i32([0]), i32(rows), 300, torch.float32)
    assert torch.equal(got[0].double(), k.permute(1, 0, 2)) and torch.equal(got[1].double(), v.permute(1, 0, 2))


@pytest.mark.parametrize("call", ["decode", "prefill"])
def test_wait_timeout_is_flagged_and_leaves_the_workspace_fit(tq, call):
    """Every other CTA (decode) or split (prefill) gives up a bounded wait: the call is flagged and returns, and the
    next one on the same workspace is exact."""
    gen = torch.Generator().manual_seed(15)
    n = 9000
    s = Setup(tq, gen, [n], 1, 16)
    s.fill([n], outliers=False)
    q = torch.randn(20, 8, D, generator=gen).bfloat16().cuda()
    run = (lambda st: s.cache.decode(q[:1], s.table, i32([n]), status=st)) if call == "decode" else (
        lambda st: s.cache.prefill(q, i32([0, 20]), i32([n - 20]), s.table, status=st))
    st = tq.new_status()
    want = run(st)
    assert st.item() == 0
    tq.set_test_stall(200000)
    try:
        run(st)
        torch.cuda.synchronize()
    finally:
        tq.set_test_stall(0)
    assert st.item() == tq.FLAG_TIMEOUT
    st = tq.new_status()
    assert torch.equal(run(st), want) and st.item() == 0
