"""64-bit definitions of the norm-and-rotation rows and of the attention over
selected blocks, written for clarity on small CPU tensors; with each value
the magnitudes that its error bound is made of."""
from __future__ import annotations

import math

import torch


def rotate_ref(n, pos, inv_freq, r0, interleaved, scale=1.0, back=False):
    """n [S, B, H, D] fp64 rotated; also |a| + |b| of each element's pair
    (|n| outside the rotated part), times scale."""
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    y, mag = n.clone(), n.abs()
    for i in range(R // 2):
        if interleaved:
            ia, ib = r0 + 2 * i, r0 + 2 * i + 1
        else:
            ia, ib = r0 + i, r0 + i + R // 2
        t = pos.double() * float(inv_freq[i])
        c, s = scale * torch.cos(t)[..., None], scale * torch.sin(t)[..., None]
        if back:
            s = -s
        a, b = n[..., ia], n[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        both = scale * (a.abs() + b.abs())
        mag[..., ia], mag[..., ib] = both, both
    return y, mag


def norm_rope_ref(x, w, pos, inv_freq, r0, interleaved, eps, scale=1.0):
    n = x.double()
    if w is not None:
        n = n / torch.sqrt((n * n).mean(-1, keepdim=True) + eps) * w.double()
    return rotate_ref(n, pos, inv_freq, r0, interleaved, scale)


def norm_rope_bwd_ref(x, w, gy, pos, inv_freq, r0, interleaved, eps,
                      scale=1.0):
    """(dx, magnitude, dw, magnitude)."""
    u, mag = rotate_ref(gy.double(), pos, inv_freq, r0, interleaved, scale,
                        back=True)
    if w is None:
        return u, mag, None, None
    x, w = x.double(), w.double()
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * rstd
    dw = (u * xh).sum((0, 1, 2))
    dw_mag = (mag * xh.abs()).sum((0, 1, 2))
    g = u * w
    dx = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    gm = mag * w.abs()
    dx_mag = rstd * (gm + xh.abs() * (gm * xh.abs()).mean(-1, keepdim=True))
    return dx, dx_mag, dw, dw_mag


def row_keys(blocks, b, s, hk, pos, block, local, T):
    """Sorted keys that row (b, s) of key head hk attends to."""
    if pos < 0:
        return []
    nblk = -(-T // block)
    own = pos // block
    ids = set(range(max(0, own - local + 1), own + 1))
    if blocks is not None:
        row = blocks[b, s] if blocks.dim() == 3 else blocks[b, s, hk]
        ids |= {int(n) for n in row if 0 <= int(n) < nblk}
    return [j for n in sorted(ids) for j in range(n * block, (n + 1) * block)
            if j <= pos and j < T]


def block_attn_ref(q, k, v, blocks, block, local, scale, q_pos=None, go=None,
                   o_used=None):
    """q [S,B,H,D], k and v [T,B,Hk,D].  Returns a dict: o, lse; A_o = sum p
    |v|, X = max_j scale sum_d |q k|; with go also gq, gk, gv and the sums of
    magnitudes their tolerances need (o_used: the rounded o that the backward
    reads)."""
    S, B, H, D = q.shape
    T, _, Hk, _ = k.shape
    G = H // Hk
    q, k, v = q.double(), k.double(), v.double()
    r = dict(o=torch.zeros_like(q), A_o=torch.zeros_like(q),
             lse=torch.full((S, B, H), -math.inf, dtype=torch.float64),
             X=torch.zeros((S, B, H), dtype=torch.float64))
    if go is not None:
        go = go.double()
        for n in ("gq", "tq"):
            r[n] = torch.zeros_like(q)
        for n in ("gk", "gv", "tk", "tv"):
            r[n] = torch.zeros_like(k)
    for b in range(B):
        for s in range(S):
            pos = (0 if q_pos is None else int(q_pos[b])) + s
            for hk in range(Hk):
                js = row_keys(blocks, b, s, hk, pos, block, local, T)
                if not js:
                    continue
                hs = slice(hk * G, hk * G + G)
                kk, vv, qq = k[js, b, hk], v[js, b, hk], q[s, b, hs]
                x = scale * qq @ kk.T
                lse = torch.logsumexp(x, 1)
                p = torch.exp(x - lse[:, None])
                r["o"][s, b, hs] = p @ vv
                r["A_o"][s, b, hs] = p @ vv.abs()
                r["lse"][s, b, hs] = lse
                r["X"][s, b, hs] = (scale * qq.abs() @ kk.abs().T).amax(1)
                if go is None:
                    continue
                g = go[s, b, hs]
                o = r["o"][s, b, hs]
                dp = g @ vv.T
                ds = scale * p * (dp - (g * o).sum(1, keepdim=True))
                r["gq"][s, b, hs] = ds @ kk
                # errors of dS: its own rounding (2^-8 |dS|), the rounded o in
                # do.o (2^-8 sum |do o|), and 2^-12 of everything it is made
                # of for the fp32 sums and the exponential
                dlt = (g * o).abs().sum(1, keepdim=True)
                e = (2.0 ** -8 * ds.abs() + scale * p * (
                    2.0 ** -8 * dlt + 2.0 ** -12 * (g.abs() @ vv.abs().T + dlt)))
                r["tq"][s, b, hs] = e @ kk.abs()
                ep = p * (2.0 ** -8 + 2.0 ** -12)
                r["gk"][:, b, hk].index_add_(0, torch.tensor(js), ds.T @ qq)
                r["gv"][:, b, hk].index_add_(0, torch.tensor(js), p.T @ g)
                r["tk"][:, b, hk].index_add_(0, torch.tensor(js), e.T @ qq.abs())
                r["tv"][:, b, hk].index_add_(0, torch.tensor(js), ep.T @ g.abs())
    return r


def check_attn(r, o, lse):
    """o: the weights' rounding to bf16 (2^-8 of A_o), the result's (2^-8 of
    |o|) and 2^-12 of A_o for fp32 sums and the exponential; lse: 2^-15 of
    one plus the largest score's magnitude.  Empty rows exactly."""
    o, lse = o.double().cpu(), lse.double().cpu()
    tol = (2.0 ** -8 + 2.0 ** -12) * r["A_o"] + 2.0 ** -8 * r["o"].abs() + 1e-30
    err = (o - r["o"]).abs()
    assert bool((err <= tol).all()), f"o off by {(err / tol).max():.3g} tol"
    empty = r["lse"] == -math.inf
    assert bool((lse[empty] == -math.inf).all())
    assert bool((o[empty] == 0).all())
    d = (lse - r["lse"]).abs()[~empty]
    t = (2.0 ** -15 * (1 + r["X"]))[~empty]
    assert bool((d <= t).all()), f"lse off by {(d / t).max():.3g} tol"


def check_grads(r, gq, gk, gv):
    for name, got, tol in (("gq", gq, r["tq"]), ("gk", gk, r["tk"]),
                           ("gv", gv, r["tv"])):
        want = r[name]
        t = tol + 2.0 ** -8 * (want.abs() + tol) + 1e-30
        err = (got.double().cpu() - want).abs()
        assert bool((err <= t).all()), f"{name} off by {(err / t).max():.3g} tol"
