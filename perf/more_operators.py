"""Timed cases of a step with drafted tokens over the 8-bit paged cache.

The cache holds e4m3 codes, [num_blocks, num_kv_heads, 2 (K, V), block_size, 128], and one
power-of-two scale for each block, KV head and side, [num_blocks, num_kv_heads, 2].  A step
rotates the drafted tokens' queries and keys by their positions, writes keys and values behind
each sequence's prefix, lets every node of the tree of drafts attend over the prefix and its own
ancestors, and keeps the path that was accepted.  Four paths:

  rotary   rows of heads are rotated by their positions (or by the transpose: the gradient)
  append   new K / V rows of a ragged batch are written into the cache, the keys rotated on the
           way, and the step's queries with them
  tree     the nodes of a ragged batch of trees attend over the cache that holds them: each over
           the whole prefix and over the nodes that its row of a bit mask names
  keep     the accepted nodes' stored keys and values move up behind the prefix

`run` computes them in plain torch (fp32, rounded once); with `own` set it makes the calls of
`online_kv_cache_encode_gb300.tq` instead.
"""
import math

import torch

own = False

D = 128            # head dimension
MIN_EXP = -120     # scale exponent of a block of zeros
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the queries of one decode step, a token for each of 64 sequences
        _rotary("rotary step", 64, 32, 128, "half", "none", 16384, "bf16"),
        # a training batch's gradient of partly rotated fp32 heads, far positions of a stretched context
        _rotary("rotary gradient", 5003, 20, 64, "interleaved", "parts", 262144, "f32", transpose=True),
        # the queries of a long prompt
        _rotary("rotary 32k", 32768, 64, 128, "half", "linear", 32768, "bf16"),
        # one decode step of a serving batch: a token for each of 64 sequences, most in the middle of a block
        _append("append step", 64, 1, 2000, True, 32, 8, 16, 128, "half", "none", "bf16", fused=True),
        # trees of drafted tokens behind contexts of a window, as many KV heads as query heads
        _append("append trees", 8, 33, 4095, True, 20, 20, 32, 64, "interleaved", "parts", "f16", nodes=True),
        # a long prompt's keys and values written at once
        _append("append 32k", 1, 32768, 0, False, 0, 8, 16, 128, "half", "linear", "bf16", fused=True),
        # the smallest tree: one head over a short context, where latency counts
        _tree("tree 1k", 1, 7, 1017, False, 1, 1, 16, "bf16"),
        # a tree of 64 nodes behind a long context, grouped queries
        _tree("tree 32k", 1, 64, 32704, False, 64, 8, 16, "bf16"),
        # windows of 4096 tokens, as many KV heads as query heads
        _tree("tree heads", 8, 33, 4063, True, 20, 20, 32, "f16"),
        # a serving batch: 16 nodes for each of 64 sequences with contexts from 1K to 16K
        _tree("tree batch", 64, 16, 16368, True, 32, 8, 16, "bf16", fused=True),
        # the accepted path of a serving batch's trees
        dict(name="keep step", op="keep", batch=64, new=16, ctx=1999, ragged=True, hkv=8, bs=16),
        # long accepted paths of wide trees, many heads, larger blocks
        dict(name="keep long", op="keep", batch=32, new=700, ctx=777, ragged=True, hkv=20, bs=64),
    ]


def _rotary(name, tokens, heads, rot, layout, scaling, far, dtype, transpose=False, fused=False):
    return dict(name=name, op="rotary", batch=1, new=tokens, ctx=0, heads=heads, rot=rot, layout=layout, scaling=scaling,
                far=far, dtype=dtype, transpose=transpose, fused=fused)


def _append(name, batch, new, ctx, ragged, hq, hkv, bs, rot, layout, scaling, dtype, nodes=False, fused=False):
    return dict(name=name, op="append", batch=batch, new=new, ctx=ctx, ragged=ragged, hq=hq, hkv=hkv, bs=bs, rot=rot,
                layout=layout, scaling=scaling, far=ctx + new, dtype=dtype, nodes=nodes, fused=fused)


def _tree(name, batch, new, ctx, ragged, hq, hkv, bs, dtype, fused=False):
    return dict(name=name, op="tree", batch=batch, new=new, ctx=ctx, ragged=ragged, hq=hq, hkv=hkv, bs=bs, dtype=dtype,
                fused=fused)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "append", "tree", "tree", "keep"))
    layout, scaling = rng.choice(("half", "half", "interleaved")), rng.choice(("none", "linear", "parts"))
    rot, dtype, fused, ragged = rng.choice((32, 64, 96, 128, 128)), rng.choice(("bf16", "f16", "f32")), rng.random() < 0.5, rng.random() < 0.6
    bs, hkv = rng.choice((16, 16, 32, 64, 128)), rng.choice((1, 2, 4, 8, 8, 20))
    if op == "rotary":
        heads = rng.choice((1, 2, 5, 8, 20, 32, 64))
        tokens = _log(rng, 1, min(65536, (1 << 20) // heads))
        c = _rotary("", tokens, heads, rot, layout, scaling, _log(rng, tokens, 262144), dtype, rng.random() < 0.4, fused)
    elif op == "append":
        hq, batch = hkv * rng.choice((0, 1, 2, 4, 8)), _log(rng, 1, 64)
        new = _log(rng, 1, 32768 * 8 // (max(8, hkv) + hq) // batch)
        c = _append("", batch, new, _log(rng, 1, 4096) - 1, ragged, hq, hkv, bs, rot, layout, scaling, dtype, new < 256 and rng.random() < 0.5, fused)
    elif op == "tree":
        hq, batch, new = hkv * rng.choice((1, 2, 4, 5, 7, 8, 8, 16)), _log(rng, 1, 64), _log(rng, 1, 256)
        new = max(1, min(new, 8192 // batch, (1 << 17) // (batch * hq)))
        ctx = min(32768, 64 * 8192 * 8 // (batch * hkv), int(1.3e11 / (4 * D * hq * batch * new)))
        c = _tree("", batch, new, _log(rng, 1, max(2, ctx)) - 1, ragged, hq, hkv, bs, rng.choice(("bf16", "bf16", "f16")), fused)
    else:
        batch = _log(rng, 1, 64)
        c = dict(op="keep", batch=batch, new=_log(rng, 2, 11200 // batch), ctx=_log(rng, 1, 2048) - 1, ragged=ragged, hkv=hkv, bs=bs)
    c.pop("name", None)
    return c


def _spread(n, most, low, salt):
    """n sizes in low .. most, the same for the same case."""
    return [low + (((i + 1) * 2654435761 + salt * 40503) >> 7) % (most - low + 1) for i in range(n)]


def _ranges(case):
    """(start, new) of every sequence."""
    b, new, ctx = case["batch"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [(ctx, new)] * b
    return list(zip(_spread(b, ctx, ctx // 16, 1), [new] + _spread(b - 1, new, 1 if new == 1 else 0, 2)))


def _kept(case):
    """The accepted nodes of every sequence: a part of them for some, none for some, rising."""
    out = []
    for b, (_, n) in enumerate(_ranges(case)):
        step = 1 + (b * 2654435761 >> 9) % 4
        out.append([] if b % 7 == 3 else list(range(b % 3, n, step)))
    return out


def work(case):
    op, size = case["op"], 4 if case.get("dtype") == "f32" else 2
    if op == "rotary":
        t, h, rot = case["new"], case["heads"], case["rot"]
        return {"bytes": 2 * t * h * D * size + t * (4 + 4 * rot), "flops": 3 * t * h * rot}
    ranges, hkv, bs = _ranges(case), case["hkv"], case["bs"]
    t = sum(n for _, n in ranges)
    if op == "append":
        pages = sum(-(-(s + n) // bs) - s // bs for s, n in ranges if n) * hkv
        far = len({s + i for s, n in ranges for i in range(n)})
        return {"bytes": t * hkv * 2 * D * (1 + size) + 8 * pages + 2 * t * case["hq"] * D * size + far * 4 * case["rot"],
                "flops": t * (hkv * (5 * D + 3 * case["rot"]) + 3 * case["hq"] * case["rot"])}
    if op == "keep":
        kept = sum(len(k) for k in _kept(case))
        return {"bytes": kept * (hkv * 2 * 2 * D + 4), "flops": kept * hkv * 2 * D}
    hq = case["hq"]
    cached = sum(s + n for s, n in ranges if n)
    blocks = sum(-(-(s + n) // bs) for s, n in ranges if n)
    return {"bytes": cached * hkv * 2 * D + 8 * blocks * hkv + 2 * size * t * hq * D + t * 8 * -(-case["new"] // 64),
            "flops": 4 * D * hq * sum(n * s + n * (n + 1) // 2 for s, n in ranges)}


# --------------------------------------------------------------------------- inputs
def _pow2(e):
    """2^e of an int32 tensor, exactly (-126 <= e <= 127)."""
    return ((e + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The least e >= MIN_EXP with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = x.to(torch.int32) - 9 + (m > 0.875).to(torch.int32)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp_(min=MIN_EXP)


def _rows(gen, n, heads, spread):
    """n rows of N(0, 1) with the heads' outlier channels and a factor for each token."""
    x = torch.randn(n, heads, D, generator=gen, device="cuda")
    x *= torch.exp(0.25 * torch.randn(n, 1, 1, generator=gen, device="cuda"))
    return x.mul_(spread)


def _outliers(gen, heads):
    s = torch.ones(heads, D, device="cuda")
    s.scatter_(1, torch.rand(heads, D, generator=gen, device="cuda").argsort(1)[:, :4], 20.0)
    return s


def _scaling(case):
    """(base, kind, arguments, magnitude) of the positions' angles."""
    return {"none": (10000.0, None, (), 1.0), "linear": (10000.0, "linear", (4.0,), 1.0),
            "parts": (500000.0, "parts", (8.0, 8192, 1.0, 4.0), 1.0 + 0.1 * math.log(8.0))}[case["scaling"]]


def _frequencies(case):
    """Radians a position of every pair: base^(-2 j / rot), slowed down where the context is stretched."""
    base, kind, args, _ = _scaling(case)
    f = base ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
    if kind == "linear":
        f = f / args[0]
    elif kind == "parts":  # pairs with many turns in the original context as they are, those with few slowed down
        factor, original, low, high = args
        keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = (1 - keep) * f / factor + keep * f
    return f


def _trees(ranges, gen):
    """Every node's parent (-1: the prefix) and depth, node by node; a parent lies before its children."""
    pick = torch.rand(max(1, sum(n for _, n in ranges)), generator=gen).tolist()
    parents, depths, at = [], [], 0
    for _, n in ranges:
        p = [-1 if i == 0 or pick[at + i] < 0.1 else i - 1 - int((pick[at + i] - 0.1) * min(i, 5) / 0.9) for i in range(n)]
        d = []
        for x in p:
            d.append(d[x] + 1 if x >= 0 else 0)
        parents.append(p)
        depths += d
        at += n
    return parents, depths


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    op = case["op"]
    dtype = DTYPES.get(case.get("dtype"))
    st = dict(case=case, dtype=dtype)
    if "rot" in case:  # the angles' cosines and sines, which a program keeps for all its layers
        freq, magnitude = _frequencies(case), _scaling(case)[3]
        angle = torch.arange(case["far"], dtype=torch.float64, device="cuda")[:, None] * freq.cuda()
        st["cos"], st["sin"] = (magnitude * torch.cos(angle)).float(), (magnitude * torch.sin(angle)).float()
        if own:
            from online_kv_cache_encode_gb300 import tq
            base, kind, args, magnitude = _scaling(case)
            st["rotary"] = tq.Rotary(case["rot"], case["far"], base=base, layout=case["layout"],
                                     scaling=(kind, *args) if kind else None, magnitude=magnitude)
    if op == "rotary":
        t, h = case["new"], case["heads"]
        x = torch.randn(t, h, D, generator=gen, device="cuda").to(dtype)
        if case["fused"]:  # a slice of a fused projection's output
            x = torch.cat((x, x[:, :1], x[:, :1]), 1)[:, :h]
        st.update(x=x, positions=torch.randint(0, case["far"], (t,), generator=gen, device="cuda", dtype=torch.int32))
        return st
    hkv, bs = case["hkv"], case["bs"]
    ranges = _ranges(case)
    batch, total = len(ranges), sum(n for _, n in ranges)
    nblk = [-(-(s + n) // bs) for s, n in ranges]
    mb = max(1, max(nblk))
    num_blocks = max(1, sum(nblk)) + 3
    # every sequence's blocks lie anywhere in the pool; unused entries of the table hold -1
    order = torch.randperm(num_blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((batch, mb), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(nblk):
        table[b, :n] = order[at:at + n]
        at += n
    # the pool as the program left it: every block quantised, slots past a sequence's end among them
    pool = torch.empty(num_blocks, hkv, 2, bs, D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(num_blocks, hkv, 2, dtype=torch.float32, device="cuda")
    sk, sv = _outliers(gen, hkv), _outliers(gen, hkv)
    step = max(1, (1 << 26) // (hkv * 2 * bs * D))
    for i in range(0, num_blocks, step):
        n = min(step, num_blocks - i)
        x = torch.stack((_rows(gen, n * bs, hkv, sk), _rows(gen, n * bs, hkv, sv)), 1)
        x = x.view(n, bs, 2, hkv, D).permute(0, 3, 2, 1, 4)
        e = _exponent(x.abs().amax((3, 4)))
        pool[i:i + n] = (x * _pow2(-e)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[i:i + n] = _pow2(e)
    cu = [0]
    for _, n in ranges:
        cu.append(cu[-1] + n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    st.update(ranges=ranges, total=total, pool=pool, scales=scales, table=table, starts=i32([s for s, _ in ranges]),
              cu=i32(cu), cu_list=cu, most=max(n for _, n in ranges))
    if op == "append":
        k, v = _rows(gen, total, hkv, sk).to(dtype), _rows(gen, total, hkv, sv).to(dtype)
        q = torch.randn(total, case["hq"], D, generator=gen, device="cuda").to(dtype) if case["hq"] else None
        if case["fused"]:  # slices of a fused projection's output
            both = torch.cat((k, v) if q is None else (q, k, v), 1)
            k, v = both[:, case["hq"]:case["hq"] + hkv], both[:, case["hq"] + hkv:]
            q = both[:, :case["hq"]] if case["hq"] else None
        positions = None
        if case["nodes"]:  # a node's position is its depth in the tree, not its slot
            _, depths = _trees(ranges, host)
            first = [s for s, n in ranges for _ in range(n)]
            positions = i32([a + b for a, b in zip(first, depths)])
        st.update(k=k, v=v, q=q, positions=positions)
    if op == "tree":
        hq = case["hq"]
        q = torch.randn(total, hq, D, generator=gen, device="cuda").to(dtype)
        if case["fused"]:
            q = torch.cat((q, torch.zeros(total, 2 * hkv, D, dtype=dtype, device="cuda")), 1)[:, :hq]
        parents, _ = _trees(ranges, host)
        words, rows = -(-case["new"] // 64), []
        for p in parents:
            seen = []
            for i, x in enumerate(p):  # a node sees itself and what its parent sees
                seen.append((seen[x] if x >= 0 else 0) | 1 << i)
            rows += seen
        signed = lambda x: x - (1 << 64) if x >> 63 else x  # noqa: E731
        mask = [[signed(r >> 64 * w & (1 << 64) - 1) for w in range(words)] for r in rows]
        st.update(q=q, parents=parents, mask=torch.tensor(mask, dtype=torch.int64, device="cuda").view(total, words))
    if op == "keep":
        kept, at = _kept(case), [0]
        for k in kept:
            at.append(at[-1] + len(k))
        st.update(kept_list=kept, kept=i32([x for k in kept for x in k]), cu_kept=i32(at), kept_total=at[-1])
    if own:
        from online_kv_cache_encode_gb300 import tq
        st["cache"] = tq.Fp8Cache(num_blocks, hkv, block_size=bs, pool=pool.view(-1), scales=scales)
    return st


# --------------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        if op == "rotary":
            return st["rotary"].apply(st["x"], st["positions"], transpose=st["case"]["transpose"])
        c = st["cache"]
        if op == "append":
            q = c.append(st["k"], st["v"], st["cu"], st["starts"], st["table"], st["rotary"], positions=st["positions"], q=st["q"])
            return [st["pool"].view(torch.float8_e4m3fn), st["scales"]] + ([] if q is None else [q])
        if op == "tree":
            return c.tree(st["q"], st["cu"], st["starts"], st["table"], st["mask"])
        c.keep(st["cu_kept"], st["kept"], st["starts"], st["table"])
        return [st["pool"].view(torch.float8_e4m3fn), st["scales"]]
    return {"rotary": _run_rotary, "append": _run_append, "tree": _run_tree, "keep": _run_keep}[op](st)


def _rotate(st, x, positions, transpose=False):
    """x [T, heads, D] in fp32, its first `rot` dims rotated pair by pair."""
    x = x.float()
    c, s = (st[n][positions.long()][:, None] for n in ("cos", "sin"))
    if transpose:
        s = -s
    rot = st["case"]["rot"]
    if st["case"]["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _run_rotary(st):
    return _rotate(st, st["x"], st["positions"], st["case"]["transpose"]).to(st["dtype"])


def _places(cu, total):
    """The sequence of every packed row, and its place in it."""
    seq = torch.repeat_interleave(torch.arange(len(cu) - 1, device=cu.device), cu.diff().long(), output_size=total)
    return seq, torch.arange(total, device=cu.device) - cu[seq]


def _run_append(st):
    pool, scales, table = st["pool"], st["scales"], st["table"]
    nb, h, _, bs, _ = pool.shape
    seq, i = _places(st["cu"], st["total"])
    pos = st["starts"][seq] + i
    angle = pos if st["positions"] is None else st["positions"]
    blk, off = table[seq, (pos // bs).long()].long(), (pos % bs).long()
    x = torch.zeros(nb, 2, h, bs, D, device=pool.device)
    x[blk, 0, :, off] = _rotate(st, st["k"], angle)
    x[blk, 1, :, off] = st["v"].float()
    x = x.transpose(1, 2)
    new = torch.zeros(nb, bs, dtype=torch.bool, device=pool.device)
    new[blk, off] = True
    touched = new.any(1)
    # slots before the first new one of a touched block hold earlier positions
    old = (torch.cumsum(new, 1) == 0) & touched[:, None]
    e_old = (scales.view(torch.int32) >> 23) - 127
    e = _exponent(x.abs().amax((3, 4)))
    e = torch.where(old.any(1)[:, None, None], torch.maximum(e, e_old), e)
    e = torch.where(touched[:, None, None], e, e_old)
    code = (x * _pow2(-e)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    moved = pool.view(torch.float8_e4m3fn).float() * _pow2((e_old - e).clamp(min=-100))[..., None, None]
    moved = moved.to(torch.float8_e4m3fn).view(torch.uint8)
    pool.copy_(torch.where(new[:, None, None, :, None], code, torch.where(old[:, None, None, :, None], moved, pool)))
    scales.copy_(_pow2(e))
    out = [pool.view(torch.float8_e4m3fn), scales]
    return out if st["q"] is None else out + [_rotate(st, st["q"], angle).to(st["dtype"])]


def _run_tree(st):
    pool, scales, q, cu, starts, mask = st["pool"].view(torch.float8_e4m3fn), st["scales"], st["q"], st["cu"], st["starts"], st["mask"]
    hkv, most, n = pool.shape[1], st["most"], cu.diff()
    group, batch = q.shape[1] // hkv, len(n)
    # all sequences padded to the longest
    blocks = st["table"].clamp(min=0).long()
    kv = pool[blocks].float() * scales[blocks][..., None, None]
    kv = kv.permute(0, 2, 3, 1, 4, 5).reshape(batch, hkv, 2, -1, D)
    length = kv.shape[3]
    row = (cu[:-1, None] + torch.arange(most, device=q.device)).clamp(max=len(q) - 1)
    x = q[row].float().view(batch, most, hkv, group, D).permute(0, 2, 3, 1, 4).reshape(batch, hkv, group * most, D)
    node = torch.arange(length, device=q.device) - starts[:, None]
    word = (node >> 6).clamp(0, mask.shape[1] - 1).long()
    bit = (mask[row].gather(2, word[:, None].expand(-1, most, -1)) >> (node & 63)[:, None]) & 1
    see = (node < 0)[:, None] | (((node >= 0) & (node < n[:, None]))[:, None] & (bit != 0))
    s = (x @ kv[:, :, 0].mT / math.sqrt(D)).view(batch, hkv, group, most, length)
    s = s.masked_fill(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    w = p.sum(-1, keepdim=True)
    o = (p.view(batch, hkv, group * most, length) @ kv[:, :, 1]).view(batch, hkv, group, most, D) / torch.where(w == 0, 1.0, w)
    seq, i = _places(cu, st["total"])
    return o.permute(0, 3, 1, 2, 4)[seq, i].reshape(q.shape).to(q.dtype)


def _run_keep(st):
    pool, scales, table = st["pool"], st["scales"], st["table"]
    nb, h, _, bs, _ = pool.shape
    seq, i = _places(st["cu_kept"], st["kept_total"])
    start = st["starts"][seq]
    src, dst = start + st["kept"], start + i
    sblk, soff = table[seq, (src // bs).long()].long(), (src % bs).long()
    dblk, doff = table[seq, (dst // bs).long()].long(), (dst % bs).long()
    e_old = (scales.view(torch.int32) >> 23) - 127
    # a block's exponent: the largest of its new codes' and, where it holds earlier positions, its own
    held = torch.zeros(nb, dtype=torch.bool, device=pool.device)
    held[dblk[(i == 0) & (doff > 0)]] = True
    touched = torch.zeros_like(held)
    touched[dblk] = True
    e = torch.full_like(e_old, -1000)
    e.scatter_reduce_(0, dblk[:, None, None].expand(-1, h, 2), e_old[sblk], "amax")
    e = torch.where(held[:, None, None], torch.maximum(e, e_old), e)
    e = torch.where(touched[:, None, None], e, e_old)
    first = torch.zeros(nb, dtype=torch.long, device=pool.device)
    first[dblk[i == 0]] = doff[i == 0]
    code = pool.view(torch.float8_e4m3fn)
    moved = code[sblk, :, :, soff].float() * _pow2((e_old[sblk] - e[dblk]).clamp(min=-100))[..., None]
    moved = moved.to(torch.float8_e4m3fn).view(torch.uint8)
    fac = _pow2((e_old - e).clamp(-100, 0))[..., None, None]
    lower = (code.float() * fac).to(torch.float8_e4m3fn).view(torch.uint8)
    old = torch.arange(bs, device=pool.device)[None] < first[:, None]
    pool.copy_(torch.where(old[:, None, None, :, None], lower, pool))
    pool[dblk, :, :, doff] = moved
    scales.copy_(_pow2(e))
    return [pool.view(torch.float8_e4m3fn), scales]


# --------------------------------------------------------------------------- in 64 bits
def _two_to(e):
    """2^e in float64 from an int64 exponent, exactly."""
    return ((e + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """The nearest value of e4m3 (ties to even): 4 significant bits, steps of 2^-9 below 2^-6."""
    _, ex = torch.frexp(x.abs())
    step = _two_to((ex.to(torch.int64) - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _e4m3_value(code):
    """What the bits stand for: sign, 4 bits of exponent (bias 7), 3 bits of fraction."""
    c = code.to(torch.int64)
    ex, fr = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(ex > 0, (8 + fr) * _two_to(ex - 10), fr * 2.0 ** -9)
    return torch.where(c >= 128, -mag, mag)


def _turned(case, x, positions, sign=1):
    """x as complex pairs times magnitude * exp(i * angle)."""
    rot, half, f = case["rot"], case["layout"] == "half", _frequencies(case).to(x.device)
    y = x.double().clone()
    pair = (lambda z: (z[..., :rot // 2], z[..., rot // 2:rot])) if half else (lambda z: (z[..., 0:rot:2], z[..., 1:rot:2]))
    angle = positions.double()[:, None, None] * f
    z = torch.complex(*(p.contiguous() for p in pair(y))) * torch.polar(torch.full_like(angle, _scaling(case)[3]), sign * angle)
    for to, val in zip(pair(y), (z.real, z.imag)):
        to.copy_(val)
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        return _turned(case, st["x"], st["positions"], -1 if case["transpose"] else 1)
    bs, hkv, ranges, cu = case["bs"], case["hkv"], st["ranges"], st["cu_list"]
    pool, scales, host = st["pool"], st["scales"].double(), st["table"].cpu().tolist()
    if op == "append":
        angle = st["positions"] if st["positions"] is not None else torch.tensor(
            [s + i for s, n in ranges for i in range(n)], device="cuda")
        k, codes, at = _turned(case, st["k"], angle), _e4m3_value(pool), 0
        for b, (s, n) in enumerate(ranges):
            for j in range(s // bs, -(-(s + n) // bs)) if n else ():
                lo, hi = max(s, j * bs) - j * bs, min(s + n, (j + 1) * bs) - j * bs
                x = torch.stack((k[at:at + hi - lo], st["v"][at:at + hi - lo].double()), 1).permute(2, 1, 0, 3)
                top = x.abs().amax((2, 3))
                # the least power of two not below top / 448
                want = _two_to(torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)).to(torch.int64))
                want = torch.where(want * 448.0 < top, 2 * want, want)
                want = torch.where(want * 224.0 >= top, want / 2, want).clamp(min=2.0 ** MIN_EXP)
                if lo:
                    want = torch.maximum(want, scales[host[b][j]])
                    codes[host[b][j], :, :, :lo] = _round_e4m3(codes[host[b][j], :, :, :lo] * (scales[host[b][j]] / want)[..., None, None])
                codes[host[b][j], :, :, lo:hi] = _round_e4m3(x / want[..., None, None])
                scales[host[b][j]] = want
                at += hi - lo
        return [codes, scales] + ([] if st["q"] is None else [_turned(case, st["q"], angle)])
    if op == "keep":
        was, codes, then = _e4m3_value(pool), _e4m3_value(pool), scales.clone()
        for b, (s, _) in enumerate(ranges):
            kept = st["kept_list"][b]
            for j in range(s // bs, -(-(s + len(kept)) // bs)) if kept else ():
                lo, hi = max(s, j * bs), min(s + len(kept), (j + 1) * bs)
                src = torch.tensor([s + kept[p - s] for p in range(lo, hi)])
                of = torch.tensor([host[b][p // bs] for p in src.tolist()], device="cuda")
                x, sc = was[of, :, :, (src % bs).cuda()], scales[of]
                want = torch.maximum(sc.amax(0), scales[host[b][j]]) if lo > j * bs else sc.amax(0)
                codes[host[b][j], :, :, :lo - j * bs] = _round_e4m3(was[host[b][j], :, :, :lo - j * bs] * (scales[host[b][j]] / want)[..., None, None])
                codes[host[b][j], :, :, lo - j * bs:hi - j * bs] = _round_e4m3(x * (sc / want)[..., None]).permute(1, 2, 0, 3)
                then[host[b][j]] = want
        return [codes, then]
    group = case["hq"] // hkv
    out = torch.zeros(st["total"], hkv, group, D, dtype=torch.float64, device="cuda")
    for b, (start, n) in enumerate(ranges):
        if not n:
            continue
        see = torch.zeros(n, start + n, dtype=torch.bool)
        see[:, :start] = True
        for i, p in enumerate(st["parents"][b]):
            if p >= 0:
                see[i] = see[p]
            see[i, start + i] = True
        see = see.cuda()
        blocks = st["table"][b, :-(-(start + n) // bs)].long()
        for h in range(hkv):
            x = _e4m3_value(pool[blocks, h]) * scales[blocks, h][..., None, None]
            k, v = (x[:, i].reshape(-1, D)[:start + n] for i in (0, 1))
            q = st["q"][cu[b]:cu[b + 1], h * group:(h + 1) * group].double()
            s = torch.where(see[:, None], torch.einsum("ngd,td->ngt", q, k) * D ** -0.5, -torch.inf)
            out[cu[b]:cu[b + 1], h] = torch.softmax(s, -1) @ v
    return out.view(st["total"], case["hq"], D)
