"""Plain float64 forms of the 8-bit paged cache's operators, for the tests.

Codes are handled as their bits (0 .. 255) and e4m3 from its definition; no
part of the library or of torch's 8-bit types is used."""
import math

import torch

D = 128
MIN_EXP = -120


def two_to(e):
    """2^e in float64 from an int64 exponent, exactly."""
    return ((e + 1023) << 52).view(torch.float64)


def value_of(codes):
    """The float64 values that e4m3 bits stand for (NaN for 0x7f and 0xff)."""
    c = codes.to(torch.int64)
    ex, fr = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(ex > 0, (1 + fr / 8) * two_to(ex - 7), fr / 512)
    mag = torch.where((c & 127) == 127, torch.full_like(mag, math.nan), mag)
    return torch.where(c >= 128, -mag, mag)


_MAGNITUDES = value_of(torch.arange(127))  # increasing


def code_of(x):
    """The bits of the nearest e4m3 value (ties to the even code, beyond 448 to 448) of float64 x."""
    mags = _MAGNITUDES.to(x.device)
    a = x.abs().clamp(max=448.0).contiguous()
    hi = torch.searchsorted(mags, a).clamp(max=126)  # first magnitude >= a
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - mags[lo], mags[hi] - a
    pick = torch.where(dl < dh, lo, torch.where(dh < dl, hi, torch.where(lo % 2 == 0, lo, hi)))
    return (pick + 128 * torch.signbit(x).long()).to(torch.uint8)


def exponent(top):
    """The least e >= MIN_EXP with top <= 448 * 2^e, for a python float."""
    if top <= 0:
        return MIN_EXP
    m, x = math.frexp(top)
    return max(MIN_EXP, x - 9 + (m > 0.875))


def write(pool, scales, K, V, cu, start, table):
    """The pool [num_blocks, hkv, 2, bs, D] (uint8) and scales after a write; K, V: [T, hkv, D]."""
    pool, scales = pool.clone(), scales.clone()
    hkv, bs = pool.shape[1], pool.shape[3]
    for b, s in enumerate(start):
        n = cu[b + 1] - cu[b]
        done = 0
        while done < n:
            p = s + done
            j, off = divmod(p, bs)
            m = min(bs - off, n - done)
            blk = int(table[b][j])
            rows = slice(cu[b] + done, cu[b] + done + m)
            for h in range(hkv):
                for side, x in ((0, K), (1, V)):
                    x = x[rows, h].double()
                    fin = torch.isfinite(x)
                    e = exponent(float(x.abs()[fin].max()) if fin.any() else 0.0)
                    if off:
                        old = int(math.log2(float(scales[blk, h, side])))
                        e = max(e, old)
                        moved = value_of(pool[blk, h, side, :off]) * 2.0 ** (old - e)
                        pool[blk, h, side, :off] = code_of(moved)
                    x = torch.where(torch.isnan(x), torch.zeros_like(x), x)
                    pool[blk, h, side, off:off + m] = code_of(x * 2.0 ** -e)
                    scales[blk, h, side] = 2.0 ** e
            done += m
    return pool, scales


def stored(pool, scales, row, length):
    """Stored keys and values [hkv, length, D] (float64) of a sequence whose block-table row is `row`."""
    bs = pool.shape[3]
    blocks = torch.as_tensor(row[:-(-length // bs)], dtype=torch.long, device=pool.device)
    x = value_of(pool[blocks]) * scales[blocks].double()[..., None, None]
    x = x.permute(1, 2, 0, 3, 4).reshape(pool.shape[1], 2, -1, D)
    return x[:, 0, :length], x[:, 1, :length]


def attend(q, k, v, limits, sm_scale, keep=None, floor=1 / 32):
    """(out, spread, sharp) for q [n, hq, D] over k, v [hkv, L, D]: row i sees tokens t < limits[i] (and keep[t]).

    out = sum_t w_t v_t; spread = sum_t w_t |v_t|, what a relative error of the weights is multiplied with; sharp
    [n, hq] = max_t sum_j (|q_j| + floor max|q|) |k_tj| sm_scale over the tokens seen, what 2^-16, the relative
    rounding in a score, is multiplied with: the products' own, and 2^-16 floor of the row's largest element for
    elements far below it, which are held in fewer bits.  Rows that see nothing are zero."""
    n, hq, _ = q.shape
    hkv, L, _ = k.shape
    x = q.double().view(n, hkv, hq // hkv, D).permute(1, 2, 0, 3)
    see = torch.arange(L, device=q.device)[None, :] < torch.as_tensor(limits, device=q.device)[:, None]
    if keep is not None:
        see = see & keep[None, :]
    k = torch.where(see.any(0)[None, :, None], k, torch.zeros_like(k))
    v = torch.where(see.any(0)[None, :, None], v, torch.zeros_like(v))
    s = (x @ k[:, None].mT * sm_scale).masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True) if L else torch.full(s.shape[:-1] + (1,), -math.inf, device=q.device)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    w = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    sharp = ((x.abs() + x.abs().amax(-1, keepdim=True) * floor) @ k.abs()[:, None].mT * sm_scale).masked_fill(~see, 0.0)
    sharp = sharp.amax(-1) if L else torch.zeros(s.shape[:-1], dtype=torch.float64, device=q.device)
    back = lambda y: y.permute(2, 0, 1, 3).reshape(n, hq, D)  # noqa: E731
    return back(w @ v[:, None]), back(w @ v.abs()[:, None]), sharp.permute(2, 0, 1).reshape(n, hq)
