"""Timed cases of the 8-bit paged cache: writing it, reading it back, and attention over it.

The cache holds e4m3 codes, [num_blocks, num_kv_heads, 2 (K, V), block_size, 128], and one
power-of-two scale for each block, KV head and side, [num_blocks, num_kv_heads, 2].  Four paths:

  write    new K / V rows of a ragged batch are quantised into the sequences' blocks; a block that
           already holds earlier positions keeps the larger scale, its codes moved to it
  read     a ragged range of positions is read back as dense K / V
  decode   one query token for each sequence attends over its cached tokens
  prefill  the new tokens of a ragged batch attend causally over the cache that holds them

`run` computes them in plain torch (fp32, rounded once); with `own` set it makes the calls of
`online_kv_cache_encode_gb300.tq.Fp8Cache` instead.
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
        # one decode step of a serving batch: a token for each of 64 sequences, most in the middle of a block
        dict(name="write step", op="write", batch=64, new=1, ctx=2000, ragged=True, hq=0, hkv=8, bs=16, dtype="bf16", fused=True),
        # a ragged batch of prompts' parts at odd starts, many heads, larger blocks
        dict(name="write ragged", op="write", batch=9, new=3001, ctx=777, ragged=True, hq=0, hkv=20, bs=32, dtype="f16", fused=False),
        # a long prompt written at once
        dict(name="write 32k", op="write", batch=1, new=32768, ctx=0, ragged=False, hq=0, hkv=8, bs=16, dtype="bf16", fused=True),
        # a small dense copy in fp32, odd ranges of five sequences
        dict(name="read ragged", op="read", batch=5, new=1999, ctx=333, ragged=True, hq=0, hkv=4, bs=64, dtype="f32", fused=False),
        # a long prompt's cache handed on as dense K / V
        dict(name="read 32k", op="read", batch=1, new=32768, ctx=0, ragged=False, hq=0, hkv=8, bs=16, dtype="bf16", fused=False),
        # the smallest decode: one head over a short context, where latency counts
        dict(name="decode 1k", op="decode", batch=1, new=1, ctx=1023, ragged=False, hq=1, hkv=1, bs=16, dtype="bf16", fused=False),
        # one sequence with a long context and grouped queries
        dict(name="decode 32k", op="decode", batch=1, new=1, ctx=32767, ragged=False, hq=64, hkv=8, bs=16, dtype="bf16", fused=False),
        # a window of 4096 tokens, as many KV heads as query heads
        dict(name="decode heads", op="decode", batch=8, new=1, ctx=4095, ragged=False, hq=20, hkv=20, bs=32, dtype="f16", fused=False),
        # a serving batch with lengths from 1K to 16K
        dict(name="decode batch", op="decode", batch=64, new=1, ctx=16383, ragged=True, hq=32, hkv=8, bs=16, dtype="bf16", fused=True),
        # a short chunk behind a long context
        dict(name="prefill chunk", op="prefill", batch=1, new=64, ctx=32704, ragged=False, hq=64, hkv=8, bs=16, dtype="bf16", fused=False),
        # ragged prompts' parts, as many KV heads as query heads
        dict(name="prefill ragged", op="prefill", batch=5, new=701, ctx=1999, ragged=True, hq=20, hkv=20, bs=64, dtype="f16", fused=True),
        # a chunk of 4096 tokens late in a long prompt
        dict(name="prefill 4k", op="prefill", batch=1, new=4096, ctx=12288, ragged=False, hq=64, hkv=8, bs=16, dtype="bf16", fused=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "decode", "prefill"))
    ragged, fused, bs = rng.random() < 0.6, rng.random() < 0.5, rng.choice((16, 16, 32, 64, 128))
    hkv = rng.choice((1, 2, 4, 8, 8, 20))
    if op in ("write", "read"):
        batch = _log(rng, 1, 64)
        new = _log(rng, 1, 32768 * 8 // max(8, hkv) // batch)
        return dict(op=op, batch=batch, new=new, ctx=_log(rng, 1, 4096) - 1, ragged=ragged, hq=0, hkv=hkv, bs=bs,
                    dtype=rng.choice(("bf16", "f16", "f32")), fused=fused and op == "write")
    hq = hkv * rng.choice((1, 2, 4, 5, 7, 8, 8, 16))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if op == "decode":
        batch = _log(rng, 1, 64)
        ctx = _log(rng, 1, min(32768, 64 * 8192 * 8 // (batch * hkv))) - 1
        return dict(op=op, batch=batch, new=1, ctx=ctx, ragged=ragged, hq=hq, hkv=hkv, bs=bs, dtype=dtype, fused=fused)
    batch = _log(rng, 1, 8)
    pairs = 1.6e12 / (4 * D * hq * batch)  # (query, key) pairs of a sequence that keep the work below the largest case's
    new = _log(rng, 2, min(2048, int(math.sqrt(pairs))))
    ctx = _log(rng, 1, max(1, min(32768, int(pairs / new - new / 2)))) - 1
    return dict(op=op, batch=batch, new=new, ctx=ctx, ragged=ragged, hq=hq, hkv=hkv, bs=bs, dtype=dtype, fused=fused)


def _spread(n, most, low, salt):
    """n sizes in low .. most, the same for the same case."""
    return [low + (((i + 1) * 2654435761 + salt * 40503) >> 7) % (most - low + 1) for i in range(n)]


def _ranges(case):
    """(start, new) of every sequence."""
    b, new, ctx = case["batch"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [(ctx, new)] * b
    starts = _spread(b, ctx, ctx // 16, 1)
    news = [1] * b if case["op"] == "decode" or new == 1 else [new] + _spread(b - 1, new, 0, 2)
    return list(zip(starts, news))


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    hkv, hq, bs = case["hkv"], case["hq"], case["bs"]
    ranges = _ranges(case)
    t = sum(n for _, n in ranges)
    pages = sum(-(-(s + n) // bs) - s // bs for s, n in ranges if n) * hkv
    if case["op"] in ("write", "read"):
        return {"bytes": t * hkv * 2 * D * (1 + size) + 8 * pages, "flops": 3 * t * hkv * 2 * D}
    cached = sum(s + n for s, n in ranges if n)
    blocks = sum(-(-(s + n) // bs) for s, n in ranges if n)
    pairs = sum(n * s + n * (n + 1) // 2 for s, n in ranges)
    return {"bytes": cached * hkv * 2 * D + 8 * blocks * hkv + 2 * size * t * hq * D, "flops": 4 * D * hq * pairs}


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    hkv, hq, bs, op = case["hkv"], case["hq"], case["bs"], case["op"]
    dtype = DTYPES[case["dtype"]]
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
    starts = torch.tensor([s for s, _ in ranges], dtype=torch.int32, device="cuda")
    cu = [0]
    for _, n in ranges:
        cu.append(cu[-1] + n)
    st = dict(case=case, ranges=ranges, total=total, pool=pool, scales=scales, table=table, starts=starts, cu_list=cu,
              cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), dtype=dtype,
              lens=torch.tensor([s + n for s, n in ranges], dtype=torch.int32, device="cuda"))
    if op == "write":
        k, v = _rows(gen, total, hkv, sk).to(dtype), _rows(gen, total, hkv, sv).to(dtype)
        if case["fused"]:  # slices of a fused projection's output
            both = torch.stack((k, k, v), 1).contiguous()
            k, v = both[:, 1], both[:, 2]
        st.update(k=k, v=v)
    if op in ("decode", "prefill"):
        q = torch.randn(total, hq, D, generator=gen, device="cuda").to(dtype)
        if case["fused"]:
            q = torch.cat((q, torch.zeros(total, 2 * hkv, D, dtype=dtype, device="cuda")), 1)[:, :hq]
        st.update(q=q)
    # where each new token lies: its block, its offset there, and the touched block it is in
    blk, off, touch, touched, held = [], [], [], [], []
    if op in ("write", "read"):
        host = table.cpu().tolist()
        for b, (s, n) in enumerate(ranges):
            for j in range(s // bs, -(-(s + n) // bs)) if n else ():
                lo, hi = max(s, j * bs), min(s + n, (j + 1) * bs)
                blk += [host[b][j]] * (hi - lo)
                off += range(lo - j * bs, hi - j * bs)
                touch += [len(touched)] * (hi - lo)
                touched.append(host[b][j])
                held.append(lo - j * bs)
        t = lambda x: torch.tensor(x, dtype=torch.int64, device="cuda")  # noqa: E731
        st.update(blk=t(blk), off=t(off), touch=t(touch), touched=t(touched), held=t(held))
    if own:
        from online_kv_cache_encode_gb300 import tq
        st["cache"] = tq.Fp8Cache(num_blocks, hkv, block_size=bs, pool=pool.view(-1), scales=scales)
    return st


# --------------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        c = st["cache"]
        if op == "write":
            c.write(st["k"], st["v"], st["cu"], st["starts"], st["table"])
            return [st["pool"].view(torch.float8_e4m3fn), st["scales"]]
        if op == "read":
            return list(c.read(st["cu"], st["starts"], st["table"], st["total"], st["dtype"]))
        if op == "decode":
            return c.decode(st["q"], st["table"], st["lens"])
        return c.prefill(st["q"], st["cu"], st["starts"], st["table"])
    return {"write": _write, "read": _read, "decode": _attend, "prefill": _attend}[op](st)


def _write(st):
    pool, scales, touch, off = st["pool"], st["scales"], st["touch"], st["off"]
    n, (_, h, _, bs, _) = len(st["touched"]), pool.shape
    x = torch.zeros(n, h, 2, bs, D, device=pool.device)
    x[touch, :, 0, off] = st["k"].float()
    x[touch, :, 1, off] = st["v"].float()
    new = torch.zeros(n, bs, dtype=torch.bool, device=pool.device)
    new[touch, off] = True
    slot = torch.arange(bs, device=pool.device)
    old = slot[None, :] < st["held"][:, None]
    was = pool[st["touched"]]
    e_old = (scales[st["touched"]].view(torch.int32) >> 23) - 127
    e = _exponent(x.abs().amax((3, 4)))
    e = torch.where((st["held"] > 0)[:, None, None], torch.maximum(e, e_old), e)
    code = (x * _pow2(-e)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    moved = was.view(torch.float8_e4m3fn).float() * _pow2((e_old - e).clamp(min=-100))[..., None, None]
    moved = moved.to(torch.float8_e4m3fn).view(torch.uint8)
    code = torch.where(new[:, None, None, :, None], code, torch.where(old[:, None, None, :, None], moved, was))
    pool[st["touched"]] = code
    scales[st["touched"]] = _pow2(e)
    return [pool.view(torch.float8_e4m3fn), scales]


def _read(st):
    blk, off = st["blk"], st["off"]
    code = st["pool"].view(torch.float8_e4m3fn)
    return [(code[blk, :, i, off].float() * st["scales"][blk][:, :, i, None]).to(st["dtype"]) for i in (0, 1)]


def _attend(st):
    pool, scales, q = st["pool"].view(torch.float8_e4m3fn), st["scales"], st["q"]
    hkv, bs = pool.shape[1], pool.shape[3]
    group = q.shape[1] // hkv
    out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    for b, (start, n) in enumerate(st["ranges"]):
        if not n:
            continue
        t0, length = st["cu_list"][b], start + n
        blocks = st["table"][b, :-(-length // bs)].long()
        kv = pool[blocks].float() * scales[blocks][..., None, None]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(hkv, 2, -1, D)[:, :, :length]
        at = torch.arange(length, device=q.device)
        for h in range(0, hkv, hkv if n == 1 else 1):
            hs = slice(h, hkv if n == 1 else h + 1)
            x = q[t0:t0 + n].float().view(n, hkv, group, D)[:, hs].permute(1, 2, 0, 3)
            s = x @ kv[hs, None, 0].mT / math.sqrt(D)
            s = s.masked_fill(at[None, :] > start + torch.arange(n, device=q.device)[:, None], -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = (p @ kv[hs, None, 1]) / p.sum(-1, keepdim=True)
            out[t0:t0 + n].view(n, hkv, group, D)[:, hs] = o.permute(2, 0, 1, 3).to(q.dtype)
    return out


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


def exact(case, seed):
    st = prepare(case, seed)
    op, bs, hkv = case["op"], case["bs"], case["hkv"]
    pool, scales = st["pool"], st["scales"].double()
    if op == "write":
        codes = _e4m3_value(pool)
        host, at = st["table"].cpu().tolist(), 0
        lim = 2.0 ** MIN_EXP
        for b, (s, n) in enumerate(st["ranges"]):
            for j in range(s // bs, -(-(s + n) // bs)) if n else ():
                lo, hi = max(s, j * bs) - j * bs, min(s + n, (j + 1) * bs) - j * bs
                m = hi - lo
                x = torch.stack((st["k"][at:at + m], st["v"][at:at + m]), 1).double().permute(2, 1, 0, 3)
                top = x.abs().amax((2, 3))
                # the least power of two not below top / 448
                want = _two_to(torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)).to(torch.int64))
                want = torch.where(want * 448.0 < top, 2 * want, want)
                want = torch.where(want * 224.0 >= top, want / 2, want).clamp(min=lim)
                if lo:
                    want = torch.maximum(want, scales[host[b][j]])
                    codes[host[b][j], :, :, :lo] = _round_e4m3(codes[host[b][j], :, :, :lo] * (scales[host[b][j]] / want)[..., None, None])
                codes[host[b][j], :, :, lo:hi] = _round_e4m3(x / want[..., None, None])
                scales[host[b][j]] = want
                at += m
        return [codes, scales]
    if op == "read":
        blk, off = st["blk"], st["off"]
        out = [[], []]
        for i in (0, 1):
            for c in range(0, len(blk), 1 << 14):
                rows = _e4m3_value(pool[blk[c:c + (1 << 14)], :, i, off[c:c + (1 << 14)]])
                out[i].append(rows * scales[blk[c:c + (1 << 14)]][:, :, i, None])
        return [torch.cat(x) if x else torch.zeros(0, hkv, D, dtype=torch.float64, device="cuda") for x in out]
    group = case["hq"] // hkv
    out = torch.zeros(st["total"], hkv, group, D, dtype=torch.float64, device="cuda")
    for b, (start, n) in enumerate(st["ranges"]):
        if not n:
            continue
        blocks = st["table"][b, :-(-(start + n) // bs)].long()
        last = start + torch.arange(n, device="cuda")
        for h in range(hkv):
            x = _e4m3_value(pool[blocks, h]) * scales[blocks, h][..., None, None]
            k, v = (x[:, i].reshape(-1, D)[:start + n] for i in (0, 1))
            q = st["q"][st["cu_list"][b]:st["cu_list"][b + 1], h * group:(h + 1) * group].double()
            for g in range(group):
                p = torch.softmax(torch.where(torch.arange(start + n, device="cuda")[None] <= last[:, None],
                                              (q[:, g] @ k.T) * D ** -0.5, -torch.inf), 1)
                out[st["cu_list"][b]:st["cu_list"][b + 1], h, g] = p @ v
    return out.view(st["total"], case["hq"], D)
