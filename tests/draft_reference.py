"""Plain float64 forms of the operators for drafted tokens, for the tests: rotary positions, attention of a tree of
nodes, and keeping the accepted ones.  Codes are handled as their bits."""
import math

import torch

from tests import fp8_reference as R

D = R.D


def frequencies(rot, base=10000.0, scaling=None):
    """Radians a position of every pair, as python floats."""
    out = []
    for j in range(rot // 2):
        b = base * scaling[1] ** (rot / (rot - 2)) if scaling and scaling[0] == "base" else base
        f = b ** (-2 * j / rot)
        if scaling and scaling[0] == "linear":
            f /= scaling[1]
        if scaling and scaling[0] == "parts":
            _, factor, original, low, high = scaling
            turns = original * f / (2 * math.pi)
            t = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = (1 - t) * f / factor + t * f
        out.append(f)
    return out


def pairs(rot, layout):
    """The dims (a, b) of every pair."""
    return [(j, j + rot // 2) if layout == "half" else (2 * j, 2 * j + 1) for j in range(rot // 2)]


def rotate(x, positions, freq, layout, magnitude=1.0, transpose=False):
    """x [T, H, d] rotated in float64, and sum |products| of every element, what the roundings are multiplied with."""
    y, size = x.double().clone(), x.double().abs().clone()
    p = torch.as_tensor(positions, dtype=torch.float64)[:, None]
    for f, (a, b) in zip(freq, pairs(2 * len(freq), layout)):
        c, s = magnitude * torch.cos(p * f), magnitude * torch.sin(p * f) * (-1 if transpose else 1)
        u, v = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
        size[..., a], size[..., b] = (u * c).abs() + (v * s).abs(), (v * c).abs() + (u * s).abs()
    return y, size


def rotate_fp32(x, table, positions, layout):
    """The rotation with every product and sum rounded to fp32, as the calls document it, from a table in fp32."""
    rot = 2 * table.shape[2]
    y = x.float().clone()
    row = table[torch.as_tensor(positions, dtype=torch.long)]
    for j, (a, b) in enumerate(pairs(rot, layout)):
        c, s = row[:, 0, j, None], row[:, 1, j, None]
        u, v = x[..., a].float(), x[..., b].float()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def tree(n, gen, width=3):
    """Parents of n nodes (-1: the prefix), each before its children."""
    return [max(-1, i - 1 - int(torch.randint(0, width, (1,), generator=gen))) for i in range(n)]


def ancestors(parents):
    """[n, n]: whether node i sees node j (itself and its ancestors)."""
    n = len(parents)
    see = torch.zeros(n, n, dtype=torch.bool)
    for i, p in enumerate(parents):
        if p >= 0:
            see[i] = see[p]
        see[i, i] = True
    return see


def mask_words(sees, words):
    """int64 [sum of rows, words] of per-sequence [n, m] truth values: bit j % 64 of word j / 64."""
    rows = []
    for see in sees:
        for r in see.tolist():
            w = [0] * words
            for j, on in enumerate(r):
                if on and j < 64 * words:
                    w[j // 64] |= 1 << (j % 64)
            rows.append([x - (1 << 64) if x >> 63 else x for x in w])
    return torch.tensor(rows, dtype=torch.int64).view(-1, words)


def attend(q, k, v, see, sm_scale, floor):
    """fp8_reference.attend() with any truth values see [n, L]."""
    n, hq, _ = q.shape
    hkv, L, _ = k.shape
    x = q.double().view(n, hkv, hq // hkv, D).permute(1, 2, 0, 3)
    any_row = see.any(0)[None, :, None]
    k, v = torch.where(any_row, k, torch.zeros_like(k)), torch.where(any_row, v, torch.zeros_like(v))
    s = (x @ k[:, None].mT * sm_scale).masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    w = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    sharp = ((x.abs() + x.abs().amax(-1, keepdim=True) * floor) @ k.abs()[:, None].mT * sm_scale).masked_fill(~see, 0.0).amax(-1)
    back = lambda y: y.permute(2, 0, 1, 3).reshape(n, hq, D)  # noqa: E731
    return back(w @ v[:, None]), back(w @ v.abs()[:, None]), sharp.permute(2, 0, 1).reshape(n, hq)


def keep(pool, scales, kept, start, table):
    """The pool and scales after every sequence's kept nodes moved up; kept: a list for each sequence."""
    was, e_was = pool.clone(), torch.log2(scales.double())
    pool, scales = pool.clone(), scales.clone()
    bs = pool.shape[3]
    for b, nodes in enumerate(kept):
        s, r = start[b], 0
        while r < len(nodes):
            j, off = divmod(s + r, bs)
            m = min(bs - off, len(nodes) - r)
            blk = int(table[b][j])
            src = [(int(table[b][(s + k) // bs]), (s + k) % bs) for k in nodes[r:r + m]]
            e = torch.stack([e_was[x] for x, _ in src]).amax(0)
            if off:
                e = torch.maximum(e, e_was[blk])
                down = (2.0 ** (e_was[blk] - e))[..., None, None]
                pool[blk, :, :, :off] = R.code_of(R.value_of(was[blk, :, :, :off]) * down)
            for i, (x, slot) in enumerate(src):
                pool[blk, :, :, off + i] = R.code_of(R.value_of(was[x, :, :, slot]) * (2.0 ** (e_was[x] - e))[..., None])
            scales[blk] = (2.0 ** e).float()
            r += m
    return pool, scales
