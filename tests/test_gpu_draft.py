"""Operators for drafted tokens on the GPU: rotary positions, the append that rotates on the way, attention of trees of
drafts and keeping the accepted path, each against its float64 form, and a step of them together."""
import math

import pytest
import torch

from tests import draft_reference as DR
from tests import fp8_reference as R
from tests.test_gpu_fp8 import D, DT, PREFILL, Setup, cu_of, i32, tq  # noqa: F401

pytestmark = pytest.mark.gpu

SCALINGS = {"none": None, "linear": ("linear", 4.0), "base": ("base", 8.0), "parts": ("parts", 8.0, 8192, 1.0, 4.0)}


# --------------------------------------------------------------------------- rotary positions
def check_rotated(out, want, size):
    """cos and sin rounded to fp32 (the angle in 64 bits), two products and a sum rounded: at most 4 half steps of fp32 of
    the products' sizes (and products of the second order); then the rounding to the type, half a step of the value and
    at least half of its smallest number."""
    fi = torch.finfo(out.dtype)
    tol = 4.01 * 2.0 ** -24 * size + fi.eps / 2 * (want.abs() + 4.01 * 2.0 ** -24 * size) + fi.tiny * fi.eps
    err = (out.double().cpu() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,d,rot,scaling,magnitude", [
    (1, 1, 128, 128, "none", 1.0),
    (64, 32, 128, 128, "none", 1.0),
    (7, 5, 128, 32, "linear", 1.0),
    (33, 20, 128, 96, "parts", 1.2079),
    (9, 3, 64, 64, "base", 1.0),
    (5, 17, 80, 48, "none", 1.0),       # heads that do not divide a warp
    (3, 2, 16, 16, "none", 0.5),
    (4, 33, 576, 64, "parts", 1.0),
    (2, 4, 256, 256, "linear", 1.0),
])
def test_rotary(tq, dtype, layout, T, H, d, rot, scaling, magnitude):  # noqa: F811
    gen = torch.Generator().manual_seed(T * 100 + H)
    far = 200001
    r = tq.Rotary(rot, far, base=500000.0, layout=layout, scaling=SCALINGS[scaling], magnitude=magnitude)
    freq = DR.frequencies(rot, 500000.0, SCALINGS[scaling])
    wide = torch.randn(T, H + 3, d, generator=gen).mul(3).to(DT[dtype])
    x = wide[:, 2:2 + H]
    p = torch.randint(0, far, (T,), generator=gen)
    p[0], p[-1] = 0, far - 1
    st = tq.new_status()
    dx = wide.cuda()[:, 2:2 + H]
    for transpose in (False, True):
        want, size = DR.rotate(x, p, freq, layout, magnitude, transpose)
        out = r.apply(dx, i32(p.tolist()), transpose=transpose, status=st)
        assert out.is_contiguous() and out.dtype is DT[dtype]
        check_rotated(out, want, size)
        assert torch.equal(out[..., rot:], dx[..., rot:])
        # in place, strided out and a broadcast input give the same bytes
        own = wide.cuda()
        y = own[:, 2:2 + H]
        assert r.apply(y, i32(p.tolist()), out=y, transpose=transpose) is y and torch.equal(y, out)
        assert torch.equal(own[:, :2].cpu(), wide[:, :2]) and torch.equal(own[:, 2 + H:].cpu(), wide[:, 2 + H:])
        across = torch.empty(H, T, d, dtype=DT[dtype], device="cuda").transpose(0, 1)
        assert torch.equal(r.apply(dx, i32(p.tolist()), out=across, transpose=transpose), out)
        one = dx[:, :1].expand(T, H, d)
        assert torch.equal(r.apply(one, i32(p.tolist()), transpose=transpose), out[:, :1].expand(T, H, d))
    assert st.item() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling", list(SCALINGS))
def test_rotary_table(tq, layout, scaling):  # noqa: F811
    """Every entry of the table: the angle is rounded in 64 bits, the entry once to fp32 (and the products' 2^-52)."""
    rot, far, m = 96, 3001, 1.3
    t = tq.Rotary(rot, far, layout=layout, scaling=SCALINGS[scaling], magnitude=m).table.cpu().double()
    a = torch.arange(far, dtype=torch.float64)[:, None] * torch.tensor(DR.frequencies(rot, 10000.0, SCALINGS[scaling]), dtype=torch.float64)
    # the frequencies of two pow functions may differ by some 2^-52 of them, the angle by 3000 times that
    assert ((t[:, 0] - m * torch.cos(a)).abs() <= 2.0 ** -24 * m + 1e-10).all()
    assert ((t[:, 1] - m * torch.sin(a)).abs() <= 2.0 ** -24 * m + 1e-10).all()


def test_rotary_gradient_against_differences(tq):  # noqa: F811
    """<g, J dx> by the call, which is linear, equals <transpose(g), dx>; both in fp32 sums of 64-bit products."""
    gen = torch.Generator().manual_seed(4)
    r = tq.Rotary(64, 1000, layout="interleaved", magnitude=1.1)
    x, dx, g = (torch.randn(11, 3, D, generator=gen).cuda() for _ in range(3))
    p = torch.randint(0, 1000, (11,), generator=gen).int().cuda()
    h = 0.5
    diff = (r.apply(x + h * dx, p).double() - r.apply(x - h * dx, p).double()) / (2 * h)
    back = r.apply(g, p, transpose=True).double()
    left, right = (g.double() * diff).sum(), (back * dx.double()).sum()
    # every element is off by at most 8 half steps of fp32 of numbers below 20 (the differences' operands), random in sign:
    # their sum over 4224 elements with factors below 5 stays below the sum of their sizes
    assert abs(left - right) <= 4224 * 5 * 20 * 8 * 2.0 ** -24


def test_rotary_flags_positions_outside(tq):  # noqa: F811
    r = tq.Rotary(32, 10)
    x = torch.randn(4, 2, D).bfloat16().cuda()
    out, st = torch.full_like(x, 7), tq.new_status()
    r.apply(x, i32([9, -1, 10, 0]), out=out, status=st)
    assert st.item() == tq.FLAG_BAD_SLOT
    assert (out[1:3] == 7).all() and torch.equal(out[3], x[3]) and not torch.equal(out[0], x[0])


def test_rotary_undoes_itself_and_moves_scores_by_distance(tq):  # noqa: F811
    """Transposed after forward gives the input back; <R(p) q, R(p') k> depends on p - p' only.  fp32: some 2^-22."""
    gen = torch.Generator().manual_seed(5)
    r = tq.Rotary(128, 5000)
    q, k = (torch.randn(6, 1, D, generator=gen).cuda() for _ in range(2))
    p = i32([0, 1, 17, 1000, 3999, 4000])
    back = r.apply(r.apply(q, p), p, transpose=True)
    assert (back - q).abs().max() < 8 * 2.0 ** -24 * 8
    s0 = (r.apply(q, p).double() * r.apply(k, p + 30).double()).sum(-1)
    s1 = (r.apply(q, p + 900).double() * r.apply(k, p + 930).double()).sum(-1)
    assert ((s0 - s1).abs() <= 16 * 2.0 ** -24 * (q.norm(dim=-1) * k.norm(dim=-1)).double() * 8).all()


# --------------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("bs,hkv,hq,rot,starts,news,tree", [
    (16, 1, 1, 128, [0], [1], False),
    (16, 8, 32, 128, [7] * 40, [1] * 40, False),
    (32, 2, 4, 64, [0, 5, 130, 16], [3, 0, 40, 16], False),
    (64, 3, 0, 96, [15, 127, 0, 64, 129], [1, 2, 257, 1, 128], False),
    (128, 2, 40, 32, [15, 127, 0], [130, 2, 257], True),
    (16, 4, 4, 16, [100, 31], [33, 17], True),
])
def test_append_bytes(tq, dtype, layout, bs, hkv, hq, rot, starts, news, tree):  # noqa: F811
    """Every byte of the pool and every scale is the plain write's of keys rotated in fp32; the queries are the plain
    rotation's; rows behind the last sequence stay."""
    gen = torch.Generator().manual_seed(bs * 1000 + hkv)
    s = Setup(tq, gen, [a + n for a, n in zip(starts, news)], hkv, bs)
    s.fill(starts)
    T, pad = sum(news), 3
    r = tq.Rotary(rot, 4000, layout=layout, scaling=SCALINGS["parts"])
    big = torch.randn(T + pad, 1, 1, generator=gen).mul(2).exp()  # rows of very different size
    qkv = (torch.randn(T + pad, hq + 2 * hkv, D, generator=gen) * big).to(DT[dtype])
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    cu = cu_of(news)
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(starts, news)] + [torch.zeros(pad, dtype=torch.long)])
    if tree:
        pos = torch.randint(0, 4000, (T + pad,), generator=gen)
    kr = DR.rotate_fp32(k, r.table.cpu(), pos, layout)
    want, wants = R.write(s.pool.cpu(), s.scales.cpu(), kr, v, cu, starts, s.rows)
    st = tq.new_status()
    d = qkv.cuda()
    dq, dk, dv = d[:, :hq], d[:, hq:hq + hkv], d[:, hq + hkv:]
    out = torch.full((T + pad, hq, D), 7.0, dtype=DT[dtype], device="cuda") if hq else None
    got = s.cache.append(dk, dv, i32(cu), i32(starts), s.table, r, positions=i32(pos.tolist()) if tree else None,
                         q=dq if hq else None, q_out=out, status=st)
    assert st.item() == 0 and got is out
    live = ~torch.isnan(wants)
    assert torch.equal(s.scales.cpu()[live], wants[live]) and torch.isnan(s.scales.cpu()[~live]).all()
    assert torch.equal(s.pool.cpu(), want)
    if hq:
        assert torch.equal(out[:T].cpu(), DR.rotate_fp32(q[:T], r.table.cpu(), pos[:T], layout).to(DT[dtype]))
        assert (out[T:] == 7).all()
        assert torch.equal(out[:T], r.apply(dq[:T], i32(pos[:T].tolist())))
        # again, the queries in place: the same bytes in the cache (its scales are there already), and in q
        s.cache.append(dk, dv, i32(cu), i32(starts), s.table, r, positions=i32(pos.tolist()) if tree else None, q=dq, q_out=dq)
        assert torch.equal(dq[:T], out[:T]) and torch.equal(d[T:, :hq].cpu(), qkv[T:, :hq])
        assert torch.equal(d[:, hq:].cpu(), qkv[:, hq:])
        assert torch.equal(s.pool.cpu(), R.write(want, wants, kr, v, cu, starts, s.rows)[0])


def test_append_extremes(tq):  # noqa: F811
    """Infinities and NaN (of the rotated pair), zeros, values whose rotation passes fp32, positions outside the table."""
    gen = torch.Generator().manual_seed(2)
    s = Setup(tq, gen, [16] * 4, 1, 16)
    r = tq.Rotary(64, 16)
    K = torch.randn(64, 1, D, generator=gen)
    V = torch.randn(64, 1, D, generator=gen)
    K[3, 0, 5], K[4, 0, 70], V[5, 0, 9] = math.inf, math.nan, -math.inf   # 5 is rotated with 37, 70 is not
    K[16:32] = 0
    K[34, 0, 3] = K[34, 0, 35] = torch.finfo(torch.float32).max           # at position 2: past fp32 in one of the two
    cu = cu_of([16] * 4)
    pos = [i % 16 for i in range(64)]
    kr = DR.rotate_fp32(K, r.table.cpu(), pos, "half")
    kr[50] = 0
    want, wants = R.write(s.pool.cpu(), s.scales.cpu(), kr, V, cu, [0] * 4, s.rows)
    pos[50] = 16
    st = tq.new_status()
    q = torch.randn(64, 2, D, generator=gen).cuda()
    out = torch.full_like(q, 7)
    s.cache.append(K.cuda(), V.cuda(), i32(cu), i32([0] * 4), s.table, r, positions=i32(pos), q=q, q_out=out, status=st)
    assert st.item() == tq.FLAG_NONFINITE | tq.FLAG_BAD_SLOT
    live = ~torch.isnan(wants)
    assert torch.equal(s.scales.cpu()[live], wants[live]) and torch.equal(s.pool.cpu(), want)
    assert (out[50] == 7).all() and not (out[51] == 7).any()


def test_append_without_a_place(tq):  # noqa: F811
    """Blocks outside the pool, past the table and a negative start are flagged; nothing else changes, and the queries of
    rows with a position are rotated all the same."""
    gen = torch.Generator().manual_seed(3)
    s = Setup(tq, gen, [40, 40], 2, 16)
    s.fill([10, 10])
    r = tq.Rotary(128, 100)
    k = torch.randn(60, 2, D, generator=gen).bfloat16()
    table = s.table.clone()
    table[0, 1] = s.nb
    before = s.pool.clone()
    st = tq.new_status()
    out = s.cache.append(k.cuda(), k.cuda(), i32([0, 30, 60]), i32([10, -3]), table, r, q=k.cuda(),
                         q_out=torch.full((60, 2, D), 7.0, dtype=torch.bfloat16, device="cuda"), status=st)
    assert st.item() == tq.FLAG_BAD_SLOT
    kr = DR.rotate_fp32(k, r.table.cpu(), list(range(10, 40)) + [0] * 30, "half")
    assert torch.equal(out[:30].cpu(), kr[:30].bfloat16()) and (out[30:] == 7).all()
    changed = (s.pool != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) == {s.rows[0][0], s.rows[0][2]}


# --------------------------------------------------------------------------- tree
def check_tree(out, q, k, v, see, sm_scale=1 / math.sqrt(D), weights=None):
    """test_gpu_fp8.check() with any truth values: the same roundings of weights, scores and the output.  And what is
    below every type's range: a weight is formed in fp32 against a reference at most 2^25 above the row's largest (a
    whole number of octaves, 24 above), and one below 2^-126 (fp32's smallest normal number) of the reference, 2^-101 of
    the largest weight, and so of their sum, may count as 0; an output below the type's smallest number is off by up to
    that."""
    nan = (see[:, None, :, None] & (torch.isnan(v) | torch.isnan(k).any(-1, keepdim=True))[None]).any(2)
    nan = nan.repeat_interleave(q.shape[1] // k.shape[0], 1)
    assert torch.equal(torch.isnan(out), nan)
    clean = lambda x: torch.where(torch.isnan(x), torch.zeros_like(x), x)  # noqa: E731
    want, spread, sharp = DR.attend(q, clean(k), clean(v), see, sm_scale, PREFILL)
    eps = torch.finfo(out.dtype).eps
    if weights is None:
        weights = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -12
    tol = eps / 2 * want.abs() + spread * (weights + 2.0 ** -19 + 2 * 2.0 ** -16 * sharp[..., None])
    tol = tol + (2.0 ** -25 if out.dtype == torch.float16 else 2.0 ** -134)  # subnormals
    tol = tol + see.shape[1] * 2.0 ** -101 * clean(v).abs().max()
    err = torch.where(nan, torch.zeros_like(want), (out.double() - want).abs())
    assert not torch.isinf(out).any()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


def seen(start, see):
    """Truth values over the sequence's positions: the prefix and the nodes."""
    return torch.cat((torch.ones(see.shape[0], start, dtype=torch.bool), see), 1).cuda()


def run_tree(tq, s, q, starts, news, sees, words, **kw):  # noqa: F811
    st = tq.new_status()
    out = s.cache.tree(q, i32(cu_of(news)), i32(starts), s.table, DR.mask_words(sees, words).cuda(), status=st, **kw)
    return out, st.item()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bs,hq,hkv,starts,news,kind", [
    (16, 1, 1, [0], [1], "tree"),
    (16, 1, 1, [1017], [7], "tree"),
    (16, 8, 1, [0, 100, 5, 0], [130, 17, 0, 1], "tree"),
    (32, 6, 2, [127, 128, 0, 121], [2, 300, 129, 63], "tree"),
    (64, 20, 20, [333, 1], [70, 200], "any"),
    (128, 32, 2, [500], [33], "any"),
    (16, 40, 1, [0, 900], [64, 9], "any"),
    (16, 128, 1, [250], [5], "tree"),
    (32, 7, 1, [63, 0], [40, 128], "empty"),
    (16, 64, 8, [5000], [64], "tree"),
    (16, 4, 2, [0, 0, 40], [65, 16, 3], "empty"),
])
def test_tree(tq, dtype, bs, hq, hkv, starts, news, kind):  # noqa: F811
    """Trees, any masks, rows that see nothing (zero), bits behind the nodes (no effect), masks with too few words."""
    gen = torch.Generator().manual_seed(hq * 10 + bs)
    lens = [a + n for a, n in zip(starts, news)]
    s = Setup(tq, gen, lens, hkv, bs)
    s.fill(lens)
    sees = []
    for n in news:
        if kind == "tree":
            sees.append(DR.ancestors(DR.tree(n, gen)))
        else:
            sees.append(torch.rand(n, n, generator=gen) < 0.3)
            if kind == "empty" and n:
                sees[-1][::3] = False
    T, words = sum(news), -(-max(news) // 64)
    q = torch.randn(T + 2, hq + 2, D, generator=gen).to(DT[dtype]).cuda()[:, 1:1 + hq]
    out = torch.full((T + 2, hq, D), 7.0, dtype=DT[dtype], device="cuda")
    more = [torch.cat((x, torch.ones(len(x), 64 * words + 64 - x.shape[1], dtype=torch.bool)), 1) for x in sees]
    pad = [torch.ones(2, 1, dtype=torch.bool)]
    got, flags = run_tree(tq, s, q, starts, news, more + pad, words + 1, out=out)
    assert got is out and flags == 0 and (out[T:] == 7).all()
    cu = cu_of(news)
    for b, (a, n) in enumerate(zip(starts, news)):
        if n:
            k, v = R.stored(s.pool, s.scales, s.rows[b], a + n)
            check_tree(out[cu[b]:cu[b + 1]], q[cu[b]:cu[b + 1]], k, v, seen(a, sees[b]))
            if a == 0:
                assert not out[cu[b]:cu[b + 1]][~sees[b].any(1).cuda()].any()
    exact, flags = run_tree(tq, s, q, starts, news, sees + pad, words)
    assert flags == 0 and torch.equal(exact[:T], out[:T])
    if words > 1:  # nodes behind the mask's words are seen by nobody
        few, flags = run_tree(tq, s, q, starts, news, sees + pad, 1)
        cut = [torch.cat((x[:, :64], torch.zeros_like(x[:, 64:])), 1) for x in sees]
        for b, (a, n) in enumerate(zip(starts, news)):
            if n:
                k, v = R.stored(s.pool, s.scales, s.rows[b], a + n)
                check_tree(few[cu[b]:cu[b + 1]], q[cu[b]:cu[b + 1]], k, v, seen(a, cut[b]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,batch", [(16, 8, 24), (32, 2, 24), (20, 20, 3), (8, 8, 70)])
def test_tree_of_many_units(tq, dtype, hq, hkv, batch):  # noqa: F811
    """More units than SMs, of all lengths: trees without nodes, with one, behind long prefixes and none, one with a
    negative start (flagged, its rows are zero); the same bytes again."""
    gen = torch.Generator().manual_seed(53)
    starts = torch.randint(0, 900, (batch,), generator=gen).tolist()
    news = torch.randint(0, 40, (batch,), generator=gen).tolist()
    starts[0], news[0] = 0, 150
    starts[1], news[1] = 2100, 1
    starts[2], news[2] = 40, 0
    if batch > 6:
        starts[6], news[6] = -9, 20
        news[-1] = 0
    lens = [max(a, 0) + n for a, n in zip(starts, news)]
    s = Setup(tq, gen, lens, hkv, 64)
    s.fill(lens)
    sees = [DR.ancestors(DR.tree(n, gen)) for n in news]
    T = sum(news)
    q = torch.randn(T, hq, D, generator=gen).to(DT[dtype]).cuda()
    out, flags = run_tree(tq, s, q, starts, news, sees, 3)
    assert flags == (tq.FLAG_BAD_SLOT if batch > 6 else 0)
    cu = cu_of(news)
    for b, (a, n) in enumerate(zip(starts, news)):
        if n and a < 0:
            assert not out[cu[b]:cu[b + 1]].any()
        elif n:
            k, v = R.stored(s.pool, s.scales, s.rows[b], a + n)
            check_tree(out[cu[b]:cu[b + 1]], q[cu[b]:cu[b + 1]], k, v, seen(a, sees[b]))
    assert torch.equal(run_tree(tq, s, q, starts, news, sees, 3)[0], out)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bs,hq,hkv,start,new", [(16, 5, 1, 20000, 60), (128, 7, 1, 9001, 200), (32, 3, 1, 30000, 1), (16, 33, 3, 4100, 13),
                                                 (64, 128, 2, 2047, 5)])
def test_tree_of_units_in_many_runs(tq, dtype, bs, hq, hkv, start, new):  # noqa: F811
    """Few heads and nodes behind long prefixes: a unit is cut in up to as many runs as there are SMs, groups that do not
    divide a tile, units of one row tile and of two; the same bytes again."""
    gen = torch.Generator().manual_seed(start)
    s = Setup(tq, gen, [start + new], hkv, bs)
    s.fill([start + new])
    see = DR.ancestors(DR.tree(new, gen))
    q = torch.randn(new, hq, D, generator=gen).to(DT[dtype]).cuda()
    out, flags = run_tree(tq, s, q, [start], [new], [see], -(-new // 64))
    assert flags == 0
    k, v = R.stored(s.pool, s.scales, s.rows[0], start + new)
    check_tree(out, q, k, v, seen(start, see))
    assert torch.equal(run_tree(tq, s, q, [start], [new], [see], -(-new // 64))[0], out)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,batch,empty", [(10, 2, 700, 0), (7, 1, 513, 512), (4, 2, 2600, 2100), (16, 16, 1100, 1099), (2, 1, 2000, 0)])
def test_tree_of_many_sequences(tq, dtype, hq, hkv, batch, empty):  # noqa: F811
    """Hundreds and thousands of sequences: the first `empty` and most of the others without nodes, trees that fill a tile
    among those of one node; a sequence's rows are those that it has alone."""
    gen = torch.Generator().manual_seed(batch)
    news = torch.randint(1, 9, (batch,), generator=gen)
    news[torch.rand(batch, generator=gen) < (0.8 if empty else 0.1)] = 0
    news[:empty] = 0
    news = news.tolist()
    news[-1] = 70
    starts = torch.randint(0, 200, (batch,), generator=gen).tolist()
    lens = [a + n if n else 0 for a, n in zip(starts, news)]
    s = Setup(tq, gen, [max(n, 1) for n in lens], hkv, 16)
    s.fill([max(n, 1) for n in lens])
    sees = [DR.ancestors(DR.tree(n, gen)) if n else torch.zeros(0, 0, dtype=torch.bool) for n in news]
    q = torch.randn(sum(news), hq, D, generator=gen).to(DT[dtype]).cuda()
    out, flags = run_tree(tq, s, q, starts, news, sees, 2)
    assert flags == 0
    cu = cu_of(news)
    some = [b for b in range(batch) if news[b]]
    for b in some[:20] + some[len(some) // 2:len(some) // 2 + 20] + some[-20:]:
        k, v = R.stored(s.pool, s.scales, s.rows[b], lens[b])
        check_tree(out[cu[b]:cu[b + 1]], q[cu[b]:cu[b + 1]], k, v, seen(starts[b], sees[b]))
    assert not torch.isnan(out).any() and (out != 0).any(-1).all()
    assert torch.equal(run_tree(tq, s, q, starts, news, sees, 2)[0], out)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (20, 20)])
def test_tree_that_is_a_chain_is_prefill(tq, dtype, hq, hkv):  # noqa: F811
    """Nodes in one line are a causal chunk: both calls against the same float64 form."""
    gen = torch.Generator().manual_seed(9)
    starts, news = [333, 0, 64], [50, 7, 64]
    lens = [a + n for a, n in zip(starts, news)]
    s = Setup(tq, gen, lens, hkv, 16)
    s.fill(lens)
    q = torch.randn(sum(news), hq, D, generator=gen).to(DT[dtype]).cuda()
    sees = [DR.ancestors([i - 1 for i in range(n)]) for n in news]
    out, _ = run_tree(tq, s, q, starts, news, sees, 1)
    other = s.cache.prefill(q, i32(cu_of(news)), i32(starts), s.table)
    cu = cu_of(news)
    for b, (a, n) in enumerate(zip(starts, news)):
        k, v = R.stored(s.pool, s.scales, s.rows[b], a + n)
        for x in (out, other):
            check_tree(x[cu[b]:cu[b + 1]], q[cu[b]:cu[b + 1]], k, v, seen(a, sees[b]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bs,hq,hkv,start,new", [(16, 8, 2, 0, 200), (64, 5, 1, 2900, 70), (32, 20, 20, 130, 33)])
def test_tree_nan_codes(tq, dtype, bs, hq, hkv, start, new):  # noqa: F811
    """Codes of NaN among the nodes and in the prefix: NaN in the rows that see them and in no others, also where a row
    sees a later one of two such nodes only; behind the end they reach nobody."""
    gen = torch.Generator().manual_seed(61)
    n = start + new
    s = Setup(tq, gen, [n], hkv, bs)
    s.fill([n])
    for i, node in enumerate((1, 2, new // 2, new - 2)):
        p = start + node
        s.pool[s.rows[0][p // bs], 0, 1, p % bs, (37 * (i // 2) + 3) % D] = 0x7F if i % 2 else 0xFF
    if start:
        p = start // 2
        s.pool[s.rows[0][p // bs], hkv - 1, 1, p % bs, 64:70] = 0x7F
    if hkv > 1:
        p = start + new // 3
        s.pool[s.rows[0][p // bs], 1, 0, p % bs, 9] = 0x7F
    if n % bs:
        s.pool[s.rows[0][n // bs], :, :, n % bs:] = 0x7F
    q = torch.randn(new, hq, D, generator=gen).to(DT[dtype]).cuda()
    see = torch.rand(new, new, generator=gen) < 0.3
    see[5], see[6] = False, False
    see[6, 6] = True
    out, flags = run_tree(tq, s, q, [start], [new], [see], -(-new // 64))
    assert flags == 0
    k, v = R.stored(s.pool, s.scales, s.rows[0], n)
    check_tree(out, q, k, v, seen(start, see))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq", [4, 20])
def test_tree_values_at_the_limit_that_a_row_does_not_see(tq, dtype, hq):  # noqa: F811
    """Nodes whose values are 2^128, past what bf16 holds, and keys that dominate: no trace in the rows without them."""
    gen = torch.Generator().manual_seed(63)
    start, n = 50, 60
    s = Setup(tq, gen, [start + n], 1, 16)
    K, V = (torch.randn(start + n, 1, D, generator=gen).bfloat16() for _ in range(2))
    V[start + 14:start + 30, 0, ::7] = torch.finfo(torch.bfloat16).max   # (whole blocks: nodes 14 .. 29)
    K[start + 14:start + 30] *= 2.0 ** 60
    p, sc = R.write(s.pool.cpu(), s.scales.cpu(), K, V, [0, start + n], [0], s.rows)
    s.pool.copy_(p)
    s.scales.copy_(sc)
    see = DR.ancestors(DR.tree(n, gen))
    see[:, 14:30] = False
    q = torch.randn(n, hq, D, generator=gen).to(DT[dtype]).cuda()
    out, _ = run_tree(tq, s, q, [start], [n], [see], 1)
    k, v = R.stored(s.pool, s.scales, s.rows[0], start + n)
    check_tree(out, q, k, v, seen(start, see))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,start,new", [(1, 1, 1017, 7), (8, 2, 300, 20), (4, 4, 3000, 3)])
def test_tree_of_a_small_call_keeps_its_weights(tq, dtype, hq, hkv, start, new):  # noqa: F811
    """Few rows: weights and their remainders, both rounded to bf16, off by 2^-9 * 2^-9 at most (2^-17 with the sum's
    fp32 roundings in proportion), also where values of other sizes cancel."""
    gen = torch.Generator().manual_seed(65)
    s = Setup(tq, gen, [start + new], hkv, 16)
    s.fill([start + new])
    see = DR.ancestors(DR.tree(new, gen))
    q = (2 * torch.randn(new, hq, D, generator=gen)).to(DT[dtype]).cuda()
    out, flags = run_tree(tq, s, q, [start], [new], [see], 1)
    assert flags == 0
    k, v = R.stored(s.pool, s.scales, s.rows[0], start + new)
    check_tree(out, q, k, v, seen(start, see), weights=2.0 ** -17)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq", [2, 5])
def test_tree_rows_that_see_only_low_scores_behind_the_first_tile(tq, dtype, hq):  # noqa: F811
    """Rows that see nothing in the first 128 positions and scores of -180 and less behind them: their weights are as
    good as any."""
    gen = torch.Generator().manual_seed(64)
    n = 270
    s = Setup(tq, gen, [n], 1, 16)
    signs = torch.where(torch.rand(D, generator=gen) < 0.5, -1.0, 1.0)
    K, V = -4 * signs.expand(n, 1, D).bfloat16(), torch.randn(n, 1, D, generator=gen).bfloat16()
    p, sc = R.write(s.pool.cpu(), s.scales.cpu(), K, V, [0, n], [0], s.rows)
    s.pool.copy_(p)
    s.scales.copy_(sc)
    see = torch.rand(n, n, generator=gen) < 0.3
    see[1::2, :129 + n // 8] = False
    see[5] = False
    q = (4 * signs + torch.randn(n, hq, D, generator=gen) / 4).to(DT[dtype]).cuda()
    out, flags = run_tree(tq, s, q, [0], [n], [see], -(-n // 64))
    k, v = R.stored(s.pool, s.scales, s.rows[0], n)
    check_tree(out, q, k, v, seen(0, see))
    assert flags == 0 and not out[5].any() and (out[torch.arange(n) != 5] != 0).any(-1).all()


@pytest.mark.parametrize("hq", [8, 60])
def test_tree_nonfinite_query_and_scales(tq, hq):  # noqa: F811
    """A NaN or an infinity in a query row makes its own row NaN; scores of both signs and sizes; sm_scale."""
    gen = torch.Generator().manual_seed(6)
    s = Setup(tq, gen, [300], 1, 16)
    s.fill([300])
    see = DR.ancestors(DR.tree(20, gen))
    q = torch.randn(20, hq, D, generator=gen).bfloat16().cuda()
    q[3] *= 2.0 ** -60
    q[4] *= 30
    good, _ = run_tree(tq, s, q, [280], [20], [see], 1, sm_scale=0.3)
    k, v = R.stored(s.pool, s.scales, s.rows[0], 300)
    check_tree(good, q, k, v, seen(280, see), 0.3)
    bad = q.clone()
    bad[2, 2, 7], bad[9, 5, 9] = math.nan, math.inf
    out, _ = run_tree(tq, s, bad, [280], [20], [see], 1, sm_scale=0.3)
    rest = torch.ones(20, hq, dtype=torch.bool)
    rest[2, 2] = rest[9, 5] = False
    assert torch.equal(out[rest.cuda()], good[rest.cuda()]) and torch.isnan(out[~rest.cuda()]).all()


def test_tree_bad_blocks_are_skipped(tq):  # noqa: F811
    """A block outside the pool and nodes past the table are flagged and seen by nobody."""
    gen = torch.Generator().manual_seed(7)
    s = Setup(tq, gen, [100], 2, 16)
    s.fill([100])
    see = torch.ones(30, 30, dtype=torch.bool)
    q = torch.randn(30, 4, D, generator=gen).half().cuda()
    k, v = R.stored(s.pool, s.scales, s.rows[0], 100)
    for row, gone in (([*s.rows[0][:2], s.nb, *s.rows[0][3:]], range(32, 48)), (s.rows[0][:5], range(80, 100))):
        st = tq.new_status()
        out = s.cache.tree(q, i32([0, 30]), i32([70]), i32([row]), DR.mask_words([see], 1).cuda(), status=st)
        assert st.item() == tq.FLAG_BAD_SLOT
        cut = seen(70, see)
        cut[:, list(gone)] = False
        check_tree(out, q, k, v, cut)


# --------------------------------------------------------------------------- keep
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("hkv,starts,news,kept", [
    (1, [0], [1], [[0]]),
    (2, [5, 16, 0, 130], [20, 7, 40, 3], [[0, 3, 19], [], [1, 2, 39], [2]]),
    (3, [15, 0, 255], [300, 290, 5], [list(range(0, 300, 2)), list(range(290)), [1, 2, 3, 4]]),
    (8, [7] * 30, [16] * 30, [[0, 2, 5, 9, 15][:b % 6] for b in range(30)]),
])
def test_keep_bytes(tq, bs, hkv, starts, news, kept):  # noqa: F811
    """Every byte of the pool and every scale, blocks with scales many octaves apart and codes that become subnormal."""
    gen = torch.Generator().manual_seed(bs + hkv)
    lens = [a + n for a, n in zip(starts, news)]
    s = Setup(tq, gen, lens, hkv, bs)
    s.fill(lens)
    live = ~torch.isnan(s.scales)
    s.scales[live] *= torch.pow(2.0, torch.randint(-9, 10, (int(live.sum()),), generator=gen).float()).cuda()
    pool = s.pool & 0x7E | torch.randint(0, 2, s.pool.shape, generator=gen).to(torch.uint8).cuda() * 128  # (no NaN codes)
    s.pool.copy_(pool)
    want, wants = DR.keep(s.pool.cpu(), s.scales.cpu(), kept, starts, s.rows)
    st = tq.new_status()
    s.cache.keep(i32(cu_of([len(k) for k in kept])), i32([x for k in kept for x in k]), i32(starts), s.table, status=st)
    assert st.item() == 0
    ok = ~torch.isnan(wants)
    assert torch.equal(s.scales.cpu()[ok], wants[ok]) and torch.isnan(s.scales.cpu()[~ok]).all()
    assert torch.equal(s.pool.cpu(), want)


def test_keep_nan_codes_stay_nan(tq):  # noqa: F811
    gen = torch.Generator().manual_seed(1)
    s = Setup(tq, gen, [40], 1, 16)
    s.fill([40])
    s.scales[s.rows[0][2]] *= 2.0 ** -3   # where node 30 comes from
    s.pool[s.rows[0][2], 0, 1, 3, 5] = 0xFF
    s.cache.keep(i32([0, 2]), i32([0, 30]), i32([5]), s.table)
    k, v = R.stored(s.pool, s.scales, s.rows[0], 7)
    assert torch.isnan(v[0, 6, 5]) and torch.isnan(v).sum() == 1 and not torch.isnan(k).any()


def test_keep_bad_rows_are_skipped(tq):  # noqa: F811
    """Kept rows below their place, negative ones, sources and places outside: flagged, the others move."""
    gen = torch.Generator().manual_seed(2)
    s = Setup(tq, gen, [64, 64, 64], 2, 16)
    s.fill([64, 64, 64])
    s.scales.nan_to_num_(1.0)
    rows = [[*s.rows[0][:3], s.nb], s.rows[1][:4], [-1, *s.rows[2][1:4]]]
    kept = [[0, 2, 40], [3, -1, 1], [5]]             # 10 + 40 lies in the bad block; -1 and 1 < 2; block 0 of the third
    want, wants = s.pool.cpu(), s.scales.cpu()
    want, wants = DR.keep(want, wants, [[0, 2], [3], []], [10, 4, 0], s.rows)
    st = tq.new_status()
    s.cache.keep(i32([0, 3, 6, 7]), i32([x for k in kept for x in k]), i32([10, 4, 0]), i32(rows), status=st)
    assert st.item() == tq.FLAG_BAD_SLOT
    assert torch.equal(s.scales.cpu(), wants) and torch.equal(s.pool.cpu(), want)
    st, before = tq.new_status(), s.pool.clone()
    s.cache.keep(i32([0, 1, 1, 1]), i32([3]), i32([-1, 0, 0]), s.table, status=st)
    assert st.item() == tq.FLAG_BAD_SLOT and torch.equal(s.pool, before)


# --------------------------------------------------------------------------- together
def draft_step(s, r, qkv, hq, hkv, cu, starts, pos, mask):
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    q = s.cache.append(k, v, cu, starts, s.table, r, positions=pos, q=q)
    return q, s.cache.tree(q, cu, starts, s.table, mask)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_drafted_steps(tq, layout):  # noqa: F811
    """Prompts appended, then steps of trees: append, attention, the accepted path kept, the next step behind it."""
    gen = torch.Generator().manual_seed(8)
    lens, hkv, hq = [150, 37], 2, 8
    s = Setup(tq, gen, [n + 80 for n in lens], hkv, 16)
    r = tq.Rotary(64, 4096, layout=layout, scaling=("linear", 2.0))
    pool, scales = s.pool.cpu(), s.scales.cpu()
    qkv = torch.randn(sum(lens), hq + 2 * hkv, D, generator=gen).bfloat16()
    cu, done = cu_of(lens), [0, 0]
    for step in range(4):
        news = lens if step == 0 else [19, 12]
        cu = cu_of(news)
        qkv = torch.randn(sum(news), hq + 2 * hkv, D, generator=gen).bfloat16()
        parents = [[i - 1 for i in range(n)] if step == 0 else DR.tree(n, gen) for n in news]
        sees = [DR.ancestors(p) for p in parents]
        depth = [int(see[i].sum()) - 1 for see in sees for i in range(len(see))]
        pos = [done[0 if t < news[0] else 1] + d for t, d in enumerate(depth)]
        pool, scales = R.write(pool, scales, DR.rotate_fp32(qkv[:, hq:hq + hkv], r.table.cpu(), pos, layout),
                               qkv[:, hq + hkv:], cu, done, s.rows)
        q, out = draft_step(s, r, qkv.cuda(), hq, hkv, i32(cu), i32(done), i32(pos), DR.mask_words(sees, 3).cuda())
        assert torch.equal(q.cpu(), DR.rotate_fp32(qkv[:, :hq], r.table.cpu(), pos, layout).bfloat16())
        assert torch.equal(s.pool.cpu(), pool)
        for b, n in enumerate(news):
            kk, vv = R.stored(s.pool, s.scales, s.rows[b], done[b] + n)
            check_tree(out[cu[b]:cu[b + 1]], q[cu[b]:cu[b + 1]], kk, vv, seen(done[b], sees[b]))
        kept = []
        for b, n in enumerate(news):
            kept.append(list(range(n)) if step == 0 else sees[b][n - 1 - b].nonzero().flatten().tolist())
        pool, scales = DR.keep(pool, scales, kept, done, s.rows)
        s.cache.keep(i32(cu_of([len(k) for k in kept])), i32([x for k in kept for x in k]), i32(done), s.table)
        assert torch.equal(s.pool.cpu(), pool)
        done = [d + len(k) for d, k in zip(done, kept)]


def test_captured_steps(tq):  # noqa: F811
    """A step captured once and replayed with other rows, starts, masks, positions and kept paths; the results are the
    eager calls'."""
    gen = torch.Generator().manual_seed(10)
    hkv, hq, T, lens = 2, 16, 24, [300, 90]
    a, b = (Setup(tq, torch.Generator().manual_seed(77), [n + 64 for n in lens], hkv, 16) for _ in range(2))
    for s in (a, b):
        s.gen = torch.Generator().manual_seed(78)
        s.fill([n + 64 for n in lens])
    r = tq.Rotary(128, 1000)
    x = torch.zeros(T, hq + 2 * hkv, D, dtype=torch.bfloat16, device="cuda")
    cu, start, pos = i32([0, 16, 24]), i32(lens), i32([0] * T)
    mask, cu_kept, kept = torch.zeros(T, 1, dtype=torch.int64, device="cuda"), i32([0, 0, 0]), i32([0] * T)

    def step(s):
        q, out = draft_step(s, r, x, hq, hkv, cu, start, pos, mask)
        s.cache.keep(cu_kept, kept, start, s.table)
        return q, out

    step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(b)
    step(a)
    step(a)
    for cut, at, keep in (([16, 24], [300, 90], [[0, 3, 7], [1]]), ([1, 2], [303, 91], [[0], [0]]), ([0, 24], [7, 60], [[], [0, 5, 23]])):
        x.copy_(torch.randn(x.shape, generator=gen))
        cu.copy_(i32([0] + cut))
        start.copy_(i32(at))
        pos.copy_(i32([at[0 if t < cut[0] else 1] + t % 5 for t in range(T)]))
        sees = [DR.ancestors(DR.tree(n, gen)) for n in (cut[0], cut[1] - cut[0], T - cut[1])]
        mask.copy_(DR.mask_words(sees, 1))
        cu_kept.copy_(i32(cu_of([len(k) for k in keep])))
        kept[:sum(map(len, keep))] = i32([n for k in keep for n in k])
        graph.replay()
        want = step(a)
        assert all(torch.equal(u[:cut[1]], w[:cut[1]]) for u, w in zip(got, want))
        assert torch.equal(a.pool, b.pool) and torch.equal(a.scales.nan_to_num(9), b.scales.nan_to_num(9))


def test_two_streams_at_once(tq):  # noqa: F811
    """Trees of one cache on two streams without waiting for one another, appends into different sequences beside them."""
    gen = torch.Generator().manual_seed(11)
    lens = [3000, 1700]
    s = Setup(tq, gen, [n + 32 for n in lens], 1, 16)
    s.fill([n + 32 for n in lens])
    q = torch.randn(20, 8, D, generator=gen).bfloat16().cuda()
    mask = DR.mask_words([DR.ancestors(DR.tree(20, gen))], 1).cuda()
    args = [(i32([0, 20]), i32([n]), s.table[b:b + 1].contiguous()) for b, n in enumerate(lens)]
    want = [s.cache.tree(q, *a, mask) for a in args]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append((i, s.cache.tree(q, *args[i], mask)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i, x in got)


def test_two_graphs_at_once(tq):  # noqa: F811
    """Two captured calls of one cache replayed on two streams without waiting for one another, and eager ones beside
    them; then two captured with one workspace given, in turn."""
    gen = torch.Generator().manual_seed(14)
    lens = [2500, 900]
    s = Setup(tq, gen, lens, 2, 16)
    s.fill(lens)
    q = torch.randn(30, 8, D, generator=gen).half().cuda()
    mask = DR.mask_words([DR.ancestors(DR.tree(30, gen))], 1).cuda()
    args = [(i32([0, 30]), i32([n - 30]), s.table[b:b + 1].contiguous(), mask) for b, n in enumerate(lens)]
    want = [s.cache.tree(q, *a) for a in args]
    ws = torch.zeros(tq.lib().tq_fp8_tree_workspace_bytes(s.cache._h, 30, 1, 8), dtype=torch.uint8, device="cuda")
    for given in ({}, {"workspace": ws}):
        graphs, outs = [], []
        for a in args:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append(s.cache.tree(q, *a, **given))
            graphs.append(graph)
        streams = [torch.cuda.current_stream()] * 2 if given else [torch.cuda.Stream() for _ in args]
        torch.cuda.synchronize()
        for _ in range(20):
            for graph, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    graph.replay()
            eager = [s.cache.tree(q, *a, **given) for a in args]
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) and torch.equal(e, w) for x, e, w in zip(outs, eager, want))


def test_pool_beyond_32_bits(tq):  # noqa: F811
    """Blocks whose codes lie past 4 GB of the pool: append, tree and keep."""
    gen = torch.Generator().manual_seed(12)
    hkv, bs = 8, 128
    nb = (9 << 29) // (hkv * 2 * bs * D)   # 4.5 GB
    pool = torch.zeros(nb * hkv * 2 * bs * D, dtype=torch.uint8, device="cuda")
    scales = torch.ones(nb, hkv, 2, device="cuda")
    c = tq.Fp8Cache(nb, hkv, block_size=bs, pool=pool, scales=scales)
    rows, r = [[nb - 1, 3, nb - 2]], tq.Rotary(128, 400)
    K, V = (torch.randn(300, hkv, D, generator=gen).bfloat16() for _ in range(2))
    c.append(K.cuda(), V.cuda(), i32([0, 300]), i32([0]), i32(rows), r)
    small = torch.zeros(3, hkv, 2, bs, D, dtype=torch.uint8)
    kr = DR.rotate_fp32(K, r.table.cpu(), list(range(300)), "half")
    want, wants = R.write(small, torch.ones(3, hkv, 2), kr, V, [0, 300], [0], [[2, 0, 1]])
    view = pool.view(nb, hkv, 2, bs, D)
    here = lambda: (view[[3, nb - 2, nb - 1]].cpu(), scales[[3, nb - 2, nb - 1]].cpu())  # noqa: E731
    assert all(torch.equal(x, y) for x, y in zip(here(), (want, wants)))
    k, v = R.stored(want.cuda(), wants.cuda(), [2, 0, 1], 300)
    q = torch.randn(60, 16, D, generator=gen).bfloat16().cuda()
    see = DR.ancestors(DR.tree(60, gen))
    check_tree(c.tree(q, i32([0, 60]), i32([240]), i32(rows), DR.mask_words([see], 1).cuda()), q, k, v, seen(240, see))
    c.keep(i32([0, 30]), i32(list(range(0, 60, 2))), i32([240]), i32(rows))
    assert all(torch.equal(x, y) for x, y in zip(here(), DR.keep(want, wants, [list(range(0, 60, 2))], [240], [[2, 0, 1]])))


def test_tree_wait_timeout_is_flagged_and_leaves_the_workspace_fit(tq):  # noqa: F811
    """A bounded wait gives up: the call is flagged and returns, and the next one on the same workspace is exact."""
    gen = torch.Generator().manual_seed(15)
    n = 9000
    s = Setup(tq, gen, [n], 1, 16)
    s.fill([n], outliers=False)
    q = torch.randn(20, 8, D, generator=gen).bfloat16().cuda()
    see = DR.ancestors(DR.tree(20, gen))
    want, flags = run_tree(tq, s, q, [n - 20], [20], [see], 1)
    assert flags == 0
    tq.set_test_stall(200000)
    try:
        _, flags = run_tree(tq, s, q, [n - 20], [20], [see], 1)
        torch.cuda.synchronize()
    finally:
        tq.set_test_stall(0)
    assert flags == tq.FLAG_TIMEOUT
    out, flags = run_tree(tq, s, q, [n - 20], [20], [see], 1)
    assert torch.equal(out, want) and flags == 0


def test_binding_refusals(tq):  # noqa: F811
    """What the binding and the library refuse, with nothing launched; nothing to do is not an error."""
    s = Setup(tq, torch.Generator().manual_seed(1), [40], 2, 16)
    c, cu, st, r = s.cache, i32([0, 4]), i32([0]), tq.Rotary(64, 100)
    K = torch.zeros(4, 2, D, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(4, 4, D, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(4, 1, dtype=torch.int64, device="cuda")
    p, before = i32([0, 1, 2, 3]), s.pool.clone()
    for call in (lambda: c.append(K, K, cu, st, s.table, r, positions=p.long()), lambda: c.append(K, K, cu, st, s.table, r, positions=p[:3]),
                 lambda: c.append(K, K, cu, st, s.table, r, q=q.half()), lambda: c.append(K, K, cu, st, s.table, r, q=q[:3]),
                 lambda: c.append(K, K, cu, st, s.table, r, q_out=q), lambda: c.append(K, K, cu, st, s.table, r, q=q, q_out=q[:, :2]),
                 lambda: c.append(K[:, :1], K[:, :1], cu, st, s.table, r), lambda: c.append(K, K.float(), cu, st, s.table, r),
                 lambda: c.tree(q, cu, st, s.table, m.int()), lambda: c.tree(q, cu, st, s.table, m[:3]),
                 lambda: c.tree(q, cu, st, s.table, m.cpu()), lambda: c.tree(q, cu, st, s.table, m.expand(4, 2)),
                 lambda: c.keep(cu, p.long(), st, s.table), lambda: c.keep(cu[:1], p, st, s.table),
                 lambda: r.apply(q, p.long()), lambda: r.apply(q, p[:3]), lambda: r.apply(q, p, out=q.half()),
                 lambda: r.apply(q.cpu(), p), lambda: r.apply(q.transpose(1, 2), p),
                 lambda: tq.Rotary(64, 100, frequencies=[1.0]), lambda: tq.Rotary(64, 100, table=torch.zeros(100, 64))):
        with pytest.raises((AssertionError, ValueError)):
            call()
    flat = torch.zeros(4 * 8 * D, dtype=torch.bfloat16, device="cuda")
    for call, status in ((lambda: c.tree(q.float(), cu, st, s.table, m), tq.TQ_ERR_UNSUPPORTED),
                         (lambda: c.tree(q[:, :3], cu, st, s.table, m), tq.TQ_ERR_INVALID_ARG),
                         (lambda: c.tree(q, cu, st, s.table, m[:, :0]), tq.TQ_ERR_INVALID_ARG),
                         (lambda: c.tree(q, cu, st, s.table, m, sm_scale=0.0), tq.TQ_ERR_INVALID_ARG),
                         (lambda: c.append(K, K, cu, st, s.table, tq.Rotary(256, 10)), tq.TQ_ERR_INVALID_ARG),
                         (lambda: r.apply(flat[:4 * 40].view(4, 1, 40), p), tq.TQ_ERR_INVALID_ARG),
                         (lambda: tq.Rotary(32, 100).apply(flat[:4 * 40].view(4, 1, 40), p), tq.TQ_ERR_UNSUPPORTED),
                         (lambda: r.apply(flat[:4 * 48].view(4, 1, 48), p), tq.TQ_ERR_INVALID_ARG),
                         (lambda: r.apply(flat[4:4 + 512].view(4, 1, D), p), tq.TQ_ERR_INVALID_ARG),
                         (lambda: r.apply(flat[:512].view(4, 1, D), p, out=flat[D:D + 512].view(4, 1, D)), tq.TQ_ERR_INVALID_ARG),
                         (lambda: r.apply(q, p, out=torch.empty(4, 1, D, dtype=q.dtype, device="cuda").expand(4, 4, D)), tq.TQ_ERR_INVALID_ARG),
                         (lambda: c.append(K, K, cu, st, s.table, r, q=flat[:512].view(4, 1, D), q_out=flat[D:D + 512].view(4, 1, D)),
                          tq.TQ_ERR_INVALID_ARG),
                         (lambda: tq.Rotary(24, 100), tq.TQ_ERR_UNSUPPORTED), (lambda: tq.Rotary(64, 0), tq.TQ_ERR_UNSUPPORTED),
                         (lambda: tq.Rotary(64, 9, layout="other"), tq.TQ_ERR_INVALID_ARG),
                         (lambda: tq.Rotary(64, 9, magnitude=math.nan), tq.TQ_ERR_INVALID_ARG)):
        with pytest.raises(tq.TQError) as e:
            call()
        assert e.value.status == status
    torch.cuda.synchronize()
    assert torch.equal(s.pool, before)
    none = i32([0, 0])
    assert c.append(K[:0], K[:0], none, st, s.table, r, q=q[:0]).shape == (0, 4, D)
    assert c.append(K[:0], K[:0], none, st, s.table, r) is None
    assert c.tree(q[:0], none, st, s.table, m[:0]).shape == (0, 4, D)
    assert r.apply(q[:0], p[:0]).shape == (0, 4, D)
    c.keep(none, p[:0], st, s.table)
