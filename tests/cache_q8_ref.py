"""64-bit definitions of a paged cache held in 8 bits, for small CPU tensors:
what an append writes, what a read returns, the dense keys and values that the
attention sees."""
from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn


def to_e4m3(x):
    """The nearest e4m3 value of doubles (ties to even), saturating; NaN
    stays."""
    x = x.double().clamp(-448.0, 448.0)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -200)))
    step = 2.0 ** (e.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def exp_for(top):
    """Exponent of the smallest power of two s with top <= 448 s."""
    if not top > 0:
        return -40
    m, e = math.frexp(top)
    return min(max(e - (9 if m <= 0.875 else 8), -40), 40)


def exp_of(scale):
    """The exponent that a stored scale is read with."""
    if scale != scale or abs(scale) == math.inf:
        return 40
    return -40 if scale == 0 else min(max(math.frexp(abs(scale))[1] - 1, -40),
                                      40)


def dense(cache, scale, table, group):
    """[B] of [T, Hk, D] doubles: a sequence's tokens in order."""
    page = cache.shape[1]
    out = []
    for row in table.tolist():
        parts = []
        for pg in row:
            c = cache[pg].double()
            e = torch.tensor([[exp_of(float(s)) for s in g]
                              for g in scale[pg]]).double()
            parts.append(c * (2.0 ** e).repeat_interleave(group, 0)[..., None])
        out.append(torch.cat(parts))
        assert out[-1].shape[0] == len(row) * page
    return out


def append(rows, cache, scale, table, start, count, group, slack=0.0):
    """rows [S, B, Hk, D] doubles (with their error bound `slack` per element,
    0: exact) into copies of cache and scale.  Returns (values expected as
    doubles where they are exact, tolerance on code * scale, allowed scale
    exponents {(page, group, head): set}, touched mask)."""
    S, B, Hk, D = rows.shape
    page = cache.shape[1]
    val, tol = cache.double().clone(), torch.zeros(cache.shape).double()
    touched = torch.zeros(cache.shape[:3], dtype=torch.bool)
    exps = {}
    if not isinstance(slack, torch.Tensor):
        slack = torch.full(rows.shape, float(slack)).double()
    for b in range(B):
        if start[b] < 0:
            continue
        end = start[b] + min(max(count[b], 0), S)
        p = start[b]
        while p < end:
            g0 = p // group * group
            stop = min(end, g0 + group)
            pg, off = int(table[b, g0 // page]), g0 % page
            for h in range(Hk):
                x = rows[p - start[b]:stop - start[b], b, h]
                sl = slack[p - start[b]:stop - start[b], b, h]
                fin = torch.isfinite(x)
                mag = torch.where(fin, x.abs(), 0.0)
                lo = exp_for(float((mag - sl).clamp(min=0).max()))
                hi = exp_for(float((mag + sl * fin).max()))
                old = None
                if p > g0:
                    old = exp_of(float(scale[pg, off // group, h]))
                    lo, hi = max(lo, old), max(hi, old)
                exps[pg, off // group, h] = (lo, hi, old)
                # at the larger exponent where both are possible
                half = torch.maximum(x.abs() * 2.0 ** -4,
                                     torch.full_like(x, 2.0 ** (hi - 10)))
                s = slice(off + p - g0, off + stop - g0)
                val[pg, s, h] = to_e4m3(x / 2.0 ** hi) * 2.0 ** hi
                exact = sl == 0
                tol[pg, s, h] = torch.where(exact, 0.0, 2 * half + sl)
                touched[pg, s, h] = True
                if old is not None:
                    o = slice(off, off + p - g0)
                    c = cache[pg, o, h].double()
                    val[pg, o, h] = to_e4m3(c * 2.0 ** (old - hi)) * 2.0 ** hi
                    tol[pg, o, h] = 0.0 if lo == hi else 2.0 ** (hi - 9)
                    touched[pg, o, h] = True
            p = stop
    return val, tol, exps, touched
