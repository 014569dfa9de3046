"""A paged cache held in 8 bits: the append that quantises, the read back and
the attention over it, against 64-bit definitions, and the refusals of bad
arguments.

Tolerances.  Values that come without arithmetic (v, keys without norm and
rotation) are exact: codes, scales and what is read back.  Normed and rotated
keys are off by 2^-19 of the rotated pair's magnitude in fp32 (as in the
bf16 append) before their rounding to e4m3, so a value may be its neighbour:
two half steps, 2^-4 of the value or 2^-10 of the scale each, and a scale may
be the next power of two only where the largest magnitude is that close to
448 s.  Attention: the weights' rounding to fp16 (2^-11 of A_o = sum p |v|),
2^-12 of A_o for fp32 sums and the exponential, weights that fp16 holds as
subnormals (2^-31 of the largest weight times 448 for each key), the result's
half step (2^-8 of |o|); lse: 2^-15 of one plus the largest score's magnitude.
"""
from __future__ import annotations

import math

import pytest
import torch

from tests.block_ref import block_attn_ref, norm_rope_ref, row_keys
from tests.cache_q8_ref import E4M3, append, dense, exp_of, to_e4m3

gpu = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def dsa():
    import dsa_sparse_attention_fwd_gb300 as m
    m.build()
    m.load_library()
    return m


def make_cache(pages, page, Hk, D, group, seed, heads_first=False):
    g = torch.Generator().manual_seed(seed)
    shape = (pages, Hk, page, D) if heads_first else (pages, page, Hk, D)
    out = []
    for _ in range(2):
        c = (torch.randn(shape, generator=g) * 100).clamp(-448, 448).to(E4M3)
        e = torch.randint(-9, -4, (pages, page // group, Hk), generator=g)
        out += [c, 2.0 ** e.float()]
    kc, ks, vc, vs = out
    return kc, vc, ks, vs


def view(t, heads_first):
    return t.transpose(1, 2) if heads_first else t


def raw(t):
    return t.view(torch.uint8)


def weights(D, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(D, generator=g),
            1 + 0.3 * torch.randn(D, generator=g))


def inv(R):
    i = torch.arange(R // 2, dtype=torch.float64)
    return 10000.0 ** (-2 * i / R)


# ---- append ------------------------------------------------------------------

APPEND = [
    # S, B, H, Hk, D, R, r0, inter, page, pages, group, heads_first, ragged
    (1, 5, 8, 2, 128, 128, 0, False, 64, 4, 64, False, False),
    (1, 3, 2, 1, 64, 0, 0, False, 16, 4, 16, False, True),
    (2, 4, 3, 3, 16, 16, 0, True, 32, 4, 16, False, True),
    (37, 3, 4, 4, 64, 32, 32, True, 64, 3, 32, True, True),
    (200, 2, 5, 1, 128, 64, 0, False, 128, 3, 128, False, True),
    (70, 2, 0, 3, 96, 96, 0, False, 64, 4, 64, False, False),
    (150, 1, 6, 2, 256, 128, 128, True, 128, 2, 64, False, False),
    (90, 3, 4, 2, 80, 80, 0, True, 48, 5, 16, False, True),
    (33, 2, 2, 2, 192, 64, 0, False, 64, 2, 64, False, True),
    # halves that do not fall on 16-byte pieces
    (20, 2, 4, 2, 64, 24, 8, False, 32, 3, 32, False, False),
    (300, 1, 8, 8, 64, 64, 0, False, 64, 6, 64, True, False),
]


@gpu
@pytest.mark.parametrize("turned", [True, False])
@pytest.mark.parametrize("case", APPEND)
def test_append(dsa, case, turned):
    (S, B, H, Hk, D, R, r0, inter, page, pages, group, heads_first,
     ragged) = case
    g = torch.Generator().manual_seed(7)
    total = H + 2 * Hk
    qkv = torch.randn((S, B, total * D + 8), generator=g).to(BF)
    part = qkv[..., 8:].unflatten(-1, (total, D))
    q, k, v = part[:, :, :H], part[:, :, H:H + Hk], part[:, :, H + Hk:]
    P = B * pages + 3
    kc, vc, ks, vs = make_cache(P, page, Hk, D, group, 8, heads_first)
    table = torch.randperm(P, generator=g)[:B * pages].to(torch.int32)
    table = table.view(B, pages)
    start = torch.randint(0, page * pages - S + 1, (B,), generator=g)
    start[0] = start[0] // group * group     # a group that begins here
    count = None
    if ragged:
        count = torch.randint(0, S + 1, (B,), generator=g).to(torch.int32)
        count[-1] = S + 5                    # capped to S
    wq, wk = weights(D, 3)
    f = inv(R) if R else None
    if not turned:
        wk, f, R, r0 = None, None, 0, 0
    gq = qkv.cuda()[..., 8:].unflatten(-1, (total, D))
    dev = [t.cuda() for t in (kc, vc, ks, vs)]
    gkc, gvc = (view(t, heads_first) for t in dev[:2])
    with_q = H > 0 and turned
    out_q, ws = dsa.dsa_paged_append_q8(
        gq[:, :, H:H + Hk], gq[:, :, H + Hk:], gkc, gvc, dev[2], dev[3],
        table.cuda(), start.to(torch.int32).cuda(),
        count=None if count is None else count.cuda(),
        inv_freq=None if f is None else f.cuda(),
        wk=None if wk is None else wk.cuda(), eps=EPS, rot_start=r0,
        interleaved=inter, q=gq[:, :, :H] if with_q else None,
        wq=wq.cuda() if with_q else None)
    assert dsa.dsa_indexer_check(ws) == 0
    pos = start[None, :] + torch.arange(S)[:, None]
    n = [S] * B if count is None else count.tolist()
    want_k, mag = norm_rope_ref(k, wk, pos, f, r0, inter, EPS)
    slack = 2.0 ** -19 * mag if turned else 0.0
    for rows, sl, old_c, old_s, got_c, got_s in (
            (want_k, slack, kc, ks, dev[0].cpu(), dev[2].cpu()),
            (v.double(), 0.0, vc, vs, dev[1].cpu(), dev[3].cpu())):
        check_append(rows, sl, view(old_c, heads_first), old_s,
                     view(got_c, heads_first), got_s, table, start.tolist(),
                     n, group)
    if with_q:
        want, mag = norm_rope_ref(q, wq, pos, f, r0, inter, EPS)
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -19 * mag + 1e-38
        assert bool(((out_q.double().cpu() - want).abs() <= tol).all())


def check_append(rows, slack, old_c, old_s, got_c, got_s, table, start, count,
                 group):
    val, tol, exps, touched = append(rows, old_c, old_s, table, start, count,
                                     group, slack)
    want_s = old_s.clone()
    got_e = torch.zeros(got_s.shape)
    for (pg, gi, h), (lo, hi, _) in exps.items():
        s = float(got_s[pg, gi, h])
        assert lo <= exp_of(s) <= hi and s == 2.0 ** exp_of(s)
        want_s[pg, gi, h] = got_s[pg, gi, h]
        got_e[pg, gi, h] = exp_of(s)
    assert torch.equal(want_s, got_s)           # no other scale changed
    scale = (2.0 ** got_e.double()).repeat_interleave(group, 1)
    got = got_c.double() * scale[..., None]
    err = (got - val).abs()[touched]
    assert bool((err <= tol[touched]).all()), f"off by {err.max():.3g}"
    # nothing else was touched
    a, b = raw(old_c.contiguous()), raw(got_c.contiguous())
    assert torch.equal(a[~touched], b[~touched])


@gpu
@pytest.mark.parametrize("turned", [True, False])
@pytest.mark.parametrize("S,D,R,group", [
    (1, 64, 64, 16), (2, 128, 64, 64), (3, 80, 20, 16), (150, 128, 128, 128),
    (70, 256, 256, 64), (40, 16, 6, 32)])
def test_append_of_unaligned_rows(dsa, S, D, R, group, turned):
    """Rows that cannot be read in 16-byte pieces."""
    B, H, Hk, page, pages = 2, 3, 2, 128, 4
    g = torch.Generator().manual_seed(9)
    total = H + 2 * Hk
    buf = torch.randn((S, B, total * D + 3), generator=g).to(BF)
    cut = lambda t: t[..., 1:1 + total * D].unflatten(-1, (total, D))
    part = cut(buf)
    dev_part = cut(buf.cuda())
    q, k, v = part[:, :, :H], part[:, :, H:H + Hk], part[:, :, H + Hk:]
    kc, vc, ks, vs = make_cache(B * pages, page, Hk, D, group, 8)
    table = torch.randperm(B * pages, generator=g).to(torch.int32).view(B, pages)
    start = torch.tensor([group * 2 - 1, 70], dtype=torch.int32)
    wq, wk = weights(D, 3)
    f, r0 = inv(R), D - R if R < D else 0
    dev = [t.cuda() for t in (kc, vc, ks, vs)]
    kw = dict(inv_freq=f.cuda(), wk=wk.cuda(), q=dev_part[:, :, :H],
              wq=wq.cuda(), rot_start=r0) if turned else {}
    out_q, ws = dsa.dsa_paged_append_q8(
        dev_part[:, :, H:H + Hk], dev_part[:, :, H + Hk:], *dev, table.cuda(),
        start.cuda(), eps=EPS, **kw)
    assert dsa.dsa_indexer_check(ws) == 0
    pos = start[None, :] + torch.arange(S)[:, None]
    if turned:
        rows, mag = norm_rope_ref(k, wk, pos, f, r0, False, EPS)
        slack = 2.0 ** -19 * mag
        want, mag = norm_rope_ref(q, wq, pos, f, r0, False, EPS)
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -19 * mag + 1e-38
        assert bool(((out_q.double().cpu() - want).abs() <= tol).all())
    else:
        rows, slack = k.double(), 0.0
    for x, sl, i in ((rows, slack, 0), (v.double(), 0.0, 1)):
        check_append(x, sl, (kc, vc)[i], (ks, vs)[i], dev[i].cpu(),
                     dev[2 + i].cpu(), table, start.tolist(), [S] * B, group)


@gpu
def test_one_by_one_is_as_in_one_call(dsa):
    """Powers of two: the cache is the same however its tokens are cut into
    calls, but for codes that were subnormal on the way (they may be a step of
    2^-9 of the scale away)."""
    S, Hk, D, group, page = 100, 2, 64, 32, 64
    g = torch.Generator().manual_seed(1)
    k = torch.randn((S, 1, Hk, D), generator=g)
    k *= torch.exp(torch.randn((S, 1, Hk, 1), generator=g))  # scales grow
    k = k.to(BF).cuda()
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    caches = []
    for cut in ([0, S], list(range(S + 1)), [0, 7, 40, 41, 90, S]):
        dev = [t.cuda() for t in make_cache(3, page, Hk, D, group, 5)]
        for a, b in zip(cut, cut[1:]):
            start = torch.tensor([a], dtype=torch.int32, device="cuda")
            _, ws = dsa.dsa_paged_append_q8(k[a:b], k[a:b], *dev, table, start)
            assert dsa.dsa_indexer_check(ws) == 0
        caches.append(dev)
    first = caches[0]
    for other in caches[1:]:
        for i in (0, 1):
            e = first[2 + i].cpu()
            # groups that were reached
            used = dense(torch.ones((3, page, Hk, 1)), e, table.cpu(), group)
            assert torch.equal(first[2 + i][table[0].long()].view(-1, Hk)[:4],
                               other[2 + i][table[0].long()].view(-1, Hk)[:4])
            a, b = (dense(c[i].cpu(), e, table.cpu(), group)[0][:S]
                    for c in (first, other))
            near = (a - b).abs() <= 2.0 ** -9 * used[0][:S]
            assert bool(near.all())
            assert bool((a == b)[a.abs() >= 2.0 ** -5 * used[0][:S]].all())


@gpu
def test_special_values(dsa):
    """Zeros take the smallest scale, infinities saturate, a NaN stays, and
    neither counts for the scale; huge and tiny values keep to the range."""
    k = torch.zeros((32, 1, 5, 64), dtype=BF)
    k[:, 0, 1] = 1.0
    k[3, 0, 1, 5] = math.inf
    k[4, 0, 1, 6] = -math.inf
    k[5, 0, 1, 7] = math.nan
    k[:, 0, 2] = 3e38
    k[:, 0, 3] = 1e-30
    k[:, 0, 4] = math.inf
    dev = [t.cuda() for t in make_cache(2, 32, 5, 64, 32, 1)]
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, ws = dsa.dsa_paged_append_q8(k.cuda(), k.cuda(), *dev, table, start)
    assert dsa.dsa_indexer_check(ws) == 0
    kc, vc, ks, vs = (t.cpu() for t in dev)
    for c, s in ((kc, ks), (vc, vs)):
        assert s[1, 0].tolist() == [2.0 ** -40, 2.0 ** -8, 2.0 ** 40,
                                    2.0 ** -40, 2.0 ** -40]
        c = c[1].double()
        assert bool((c[:, 0] == 0).all())
        want = torch.full((32, 64), 256.0).double()
        want[3, 5], want[4, 6] = 448.0, -448.0
        got = c[:, 1]
        assert math.isnan(float(got[5, 7]))
        want[5, 7] = got[5, 7] = 0
        assert torch.equal(got, want)
        assert bool((c[:, 2] == 448).all())
        assert bool((c[:, 3] == 0).all())
        assert bool((c[:, 4] == 448).all())


@gpu
def test_append_reports_bad_pages(dsa):
    """Rows past the table and page ids outside the cache write nothing and are
    reported; a negative start and a count of zero append nothing."""
    g = torch.Generator().manual_seed(7)
    k = torch.randn((40, 6, 2, 64), generator=g).to(BF).cuda()
    dev = [t.cuda() for t in make_cache(8, 16, 2, 64, 16, 1)]
    old = [t.clone() for t in dev]
    table = torch.tensor([[0, 1, 2], [8, 3, -1], [4, 5, 6], [4, 5, 6],
                          [4, 5, 6], [4, 5, 6]], dtype=torch.int32)
    start = torch.tensor([30, 0, -1, 5, 2 ** 31 - 1, 2 ** 31 - 20],
                         dtype=torch.int32)
    count = torch.tensor([40, 40, 40, 0, 40, 3], dtype=torch.int32)
    _, ws = dsa.dsa_paged_append_q8(k, k, *dev, table.cuda(), start.cuda(),
                                    count=count.cuda())
    assert dsa.dsa_indexer_check(ws) == 6
    assert dsa.dsa_indexer_check(ws) == 0
    changed = (raw(dev[0]) != raw(old[0])).flatten(1).any(1).tolist()
    # sequence 0: positions 30 .. 47; sequence 1: its page 3 only
    assert changed == [False, True, True, True, False, False, False, False]
    # sequence 0 as if it had come alone, its earlier tokens' codes among it
    table[1], start[1], count[1] = torch.tensor([7, 3, 7]), 16, 16
    rows = torch.stack([k[:18, 0], k[16:34, 1]], 1)  # what was written
    check_append(rows.cpu().double(), 0.0, old[0].cpu(), old[2].cpu(),
                 dev[0].cpu(), dev[2].cpu(), table[:2], start[:2].tolist(),
                 [18, 16], 16)


@gpu
def test_past_32_bit_offsets(dsa):
    """A cache of more than 2^32 bytes: the last page is written, read and
    attended to where it lies."""
    page, Hk, D = 64, 8, 128
    pages = 2 ** 32 // (page * Hk * D) + 2
    kc = torch.zeros((pages, page, Hk, D), dtype=torch.uint8, device="cuda")
    kc = kc.view(E4M3)
    ks = torch.full((pages, 1, Hk), 2.0 ** -8, device="cuda")
    k = torch.randn((3, 1, Hk, D), device="cuda").to(BF)
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32,
                         device="cuda")
    start = torch.tensor([125], dtype=torch.int32, device="cuda")
    # (keys and values of one cache)
    _, ws = dsa.dsa_paged_append_q8(k, k, kc, kc, ks, ks, table, start)
    got, _, _ = dsa.dsa_paged_read_q8(kc, kc, ks, ks, table, 3, first=start,
                                      workspace=ws)
    want = to_e4m3(k.cpu().double() * 64) / 64
    assert float((got.cpu().double() - want).abs().max()) <= 2.0 ** -5
    assert bool((got != 0).any()) and not bool(raw(kc[:2]).any())
    q = torch.randn((1, 1, Hk, D), device="cuda").to(BF)
    o, _, _ = dsa.dsa_block_attn_paged_q8_fwd(
        q, kc, kc, ks, ks, table, None, 64, 0.1, q_pos=start + 2,
        local_blocks=1)
    r = block_attn_ref(q.cpu(), torch.cat([torch.zeros((61, 1, Hk, D)),
                                           got.cpu().float()]),
                       torch.cat([torch.zeros((61, 1, Hk, D)),
                                  got.cpu().float()]),
                       None, 64, 1, 0.1, q_pos=torch.tensor([63]))
    check_attn(r, o, None, 64)


# ---- read back -----------------------------------------------------------------

READ = [
    # T, B, Hk, D, page, pages, group, heads_first
    (1, 1, 1, 16, 16, 1, 16, False),
    (77, 3, 2, 64, 32, 4, 16, False),
    (130, 2, 4, 128, 128, 2, 64, True),
    (50, 2, 3, 80, 48, 3, 16, False),
    (300, 2, 1, 256, 128, 3, 128, False),
    (999, 2, 8, 64, 64, 17, 32, False),
]


@gpu
@pytest.mark.parametrize("case", READ)
def test_read(dsa, case):
    T, B, Hk, D, page, pages, group, heads_first = case
    g = torch.Generator().manual_seed(3)
    P = B * pages + 1
    kc, vc, ks, vs = make_cache(P, page, Hk, D, group, 4, heads_first)
    raw(kc).view(-1)[5] = 0x7f               # a NaN is read as one
    table = torch.randperm(P, generator=g)[:B * pages].to(torch.int32)
    table = table.view(B, pages)
    room = page * pages - T
    first = torch.randint(0, room + 1, (B,), generator=g).to(torch.int32)
    length = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    length[0] = T
    args = [view(kc.cuda(), heads_first), view(vc.cuda(), heads_first),
            ks.cuda(), vs.cuda(), table.cuda(), T]
    for f, n in ((first, length), (None, length), (first, None)):
        k, v, ws = dsa.dsa_paged_read_q8(
            *args, first=None if f is None else f.cuda(),
            length=None if n is None else n.cuda())
        assert dsa.dsa_indexer_check(ws) == 0
        for got, c, s in ((k, kc, ks), (v, vc, vs)):
            rows = dense(view(c, heads_first), s, table, group)
            want = torch.zeros((T, B, Hk, D)).double()
            for b in range(B):
                f0 = 0 if f is None else int(f[b])
                m = T if n is None else int(n[b])
                want[:m, b] = rows[b][f0:f0 + m]
            got = got.cpu().double()
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(got.nan_to_num(), want.nan_to_num())


@gpu
def test_read_reports_bad_pages(dsa):
    kc, vc, ks, vs = (t.cuda() for t in make_cache(4, 16, 2, 64, 16, 1))
    table = torch.tensor([[0, 1], [4, 2], [3, -1], [0, 1]], dtype=torch.int32)
    first = torch.tensor([0, 0, 0, -3], dtype=torch.int32).cuda()
    length = torch.tensor([32, 32, 16, 40], dtype=torch.int32).cuda()
    k, v, ws = dsa.dsa_paged_read_q8(kc, vc, ks, vs, table.cuda(), 34,
                                     first=first, length=length)
    assert dsa.dsa_indexer_check(ws) == 6
    some = (k != 0).flatten(2).any(2)
    assert some[:, 0].tolist() == [True] * 32 + [False] * 2
    assert some[:, 1].tolist() == [False] * 16 + [True] * 16 + [False] * 2
    assert some[:, 2].tolist() == [True] * 16 + [False] * 18
    assert some[:, 3].tolist() == [False] * 3 + [True] * 31
    assert torch.equal((v != 0).flatten(2).any(2), some)
    # only what is asked for: the bad pages are not looked at
    k, v, ws = dsa.dsa_paged_read_q8(
        kc, vc, ks, vs, table[2:3].contiguous().cuda(), 34,
        length=length[2:3].contiguous())
    assert dsa.dsa_indexer_check(ws) == 0


# ---- attention -----------------------------------------------------------------

def check_attn(r, o, lse, n_keys, weight_top=None):
    """(n_keys: the most that a row has)"""
    o = o.double().cpu()
    tol = ((2.0 ** -11 + 2.0 ** -12) * r["A_o"] + 2.0 ** -8 * r["o"].abs()
           + n_keys * 2.0 ** -22 * r.get("w_top", 1.0) + 1e-30)
    fin = torch.isfinite(r["o"])
    assert torch.equal(fin, torch.isfinite(o))
    err = (o - r["o"]).abs()[fin]
    assert bool((err <= tol[fin]).all()), f"o off by {(err / tol[fin]).max():.3g} tol"
    empty = r["lse"] == -math.inf
    assert bool((o[empty] == 0).all())
    if lse is not None:
        lse = lse.double().cpu()
        assert bool((lse[empty] == -math.inf).all())
        ok = torch.isfinite(r["lse"])
        assert torch.equal(ok, torch.isfinite(lse))
        d = (lse - r["lse"]).abs()[ok]
        t = (2.0 ** -15 * (1 + r["X"]))[ok]
        assert bool((d <= t).all()), f"lse off by {(d / t).max():.3g} tol"


def blocks_for(B, S, Hs, topk, nblk, seed):
    """Ids with repeats, empty entries and ids past the row's own block."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1, nblk, (B, S, Hs, topk), generator=g)
    if topk > 2:
        ids[..., 1] = ids[..., 0]
    return ids.to(torch.int32)


ATTN = [
    # S, B, H, Hk, D, block, topk, local, shared, page, group, pages
    (1, 1, 1, 1, 128, 64, 0, 99, True, 64, 64, 3),
    (1, 3, 8, 2, 128, 64, 3, 1, False, 64, 64, 6),
    (1, 2, 16, 1, 128, 64, 4, 2, True, 128, 32, 5),
    (1, 2, 24, 1, 64, 32, 5, 1, False, 32, 16, 9),
    (1, 2, 64, 1, 128, 16, 9, 2, True, 64, 64, 3),
    (1, 2, 80, 2, 64, 128, 2, 1, False, 128, 128, 4),
    (1, 4, 4, 4, 64, 16, 0, 99, True, 16, 16, 7),
    (1, 9, 12, 2, 128, 128, 0, 99, True, 256, 64, 3),
    (4, 3, 8, 2, 128, 16, 12, 3, False, 48, 16, 9),
    (5, 2, 10, 2, 64, 64, 0, 99, True, 64, 32, 5),
    (3, 2, 6, 2, 128, 32, 0, 2, True, 64, 64, 4),
    (7, 1, 64, 1, 128, 64, 2, 1, True, 64, 64, 4),
    (33, 2, 10, 2, 64, 64, 3, 2, False, 128, 64, 4),
    (70, 1, 8, 1, 128, 128, 0, 99, True, 128, 128, 3),
    (40, 2, 4, 4, 128, 32, 4, 1, True, 96, 32, 4),
    (130, 1, 16, 1, 64, 16, 8, 2, False, 64, 16, 5),
    # single tokens of many sequences
    (1, 33, 8, 2, 128, 64, 3, 1, False, 64, 64, 4),
    (1, 16, 32, 4, 64, 32, 5, 1, True, 32, 16, 7),
    (1, 22, 15, 3, 128, 16, 9, 2, False, 48, 16, 5),
    (1, 64, 16, 1, 64, 128, 2, 1, False, 128, 128, 3),
    (1, 70, 4, 1, 128, 64, 0, 99, True, 64, 64, 3),
    (2, 40, 32, 2, 64, 32, 0, 99, True, 32, 32, 5),
    (1, 3, 12, 1, 128, 32, 0, 2, True, 64, 32, 4),
]


def attn_inputs(case, seed=0, heads_first=False):
    S, B, H, Hk, D, block, topk, local, shared, page, group, pages = case
    g = torch.Generator().manual_seed(seed)
    P = B * pages + 2
    kc, vc, ks, vs = make_cache(P, page, Hk, D, group, seed + 1, heads_first)
    table = torch.randperm(P, generator=g)[:B * pages].to(torch.int32)
    table = table.view(B, pages)
    T = page * pages
    nblk = T // block
    q = torch.randn((S, B, H, D), generator=g).to(BF)
    q_pos = torch.randint(0, T - S + 1, (B,), generator=g).to(torch.int32)
    if B > 1:
        q_pos[1] = -2                        # rows without keys
    if B > 2:
        q_pos[2] = T - 1                     # the last rows past the cache
    q_pos[0] = max(0, T - S - 1)
    ids = None
    if topk:
        ids = blocks_for(B, S, 1 if shared else Hk, topk, nblk, seed + 2)
        ids = ids[:, :, 0].contiguous() if shared else ids
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, ids=ids,
                q_pos=q_pos, block=block, local=min(local, nblk), scale=0.11,
                group=group, heads_first=heads_first)


def reference(a, **over):
    a = dict(a, **over)
    hf = a["heads_first"]
    k, v = (torch.stack(dense(view(c, hf), s, a["table"], a["group"]), 1)
            for c, s in ((a["kc"], a["ks"]), (a["vc"], a["vs"])))
    r = block_attn_ref(a["q"], k, v, a["ids"], a["block"], a["local"],
                       a["scale"], q_pos=a["q_pos"])
    # the largest weight times its values' scale bounds each term that fp16
    # holds as a subnormal
    r["w_top"] = float(a["vs"].nan_to_num(0, 0, 0).max())
    return r, k.shape[0]


def call(dsa, a, **kw):
    hf = a["heads_first"]
    c = lambda t: None if t is None else t.cuda()
    return dsa.dsa_block_attn_paged_q8_fwd(
        c(a["q"]), view(c(a["kc"]), hf), view(c(a["vc"]), hf), c(a["ks"]),
        c(a["vs"]), c(a["table"]), c(a["ids"]), a["block"], a["scale"],
        q_pos=c(a["q_pos"]), local_blocks=a["local"], **kw)


@gpu
@pytest.mark.parametrize("case", ATTN)
def test_attention(dsa, case):
    a = attn_inputs(case)
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(a)
    check_attn(r, o, lse, T)
    # the same workspace again: the counts in it are back where they were
    o2, lse2, _ = call(dsa, a, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@gpu
@pytest.mark.parametrize("case", [ATTN[1], ATTN[6], ATTN[9], ATTN[12]])
def test_attention_heads_first(dsa, case):
    a = attn_inputs(case, 5, heads_first=True)
    o, lse, ws = call(dsa, a)
    r, T = reference(a)
    check_attn(r, o, lse, T)


@gpu
@pytest.mark.parametrize("case", ATTN)
def test_attention_of_unwritten_memory(dsa, case):
    """Codes and scales behind every row's position may hold anything, NaN
    among it, and so may pages that no row reaches."""
    a = attn_inputs(case, 3)
    o, lse, _ = call(dsa, a)
    S, page, group = a["q"].shape[0], a["kc"].shape[1], a["group"]
    T = page * a["table"].shape[1]
    clean = {n: a[n].clone() for n in ("kc", "vc", "ks", "vs")}
    used = set(a["table"].view(-1).tolist())
    for pg in range(a["kc"].shape[0]):
        if pg not in used:
            raw(a["kc"])[pg] = 0x7f
            raw(a["vc"])[pg] = 0xff
            a["ks"][pg] = a["vs"][pg] = math.nan
    for b, row in enumerate(a["table"].tolist()):
        last = min(int(a["q_pos"][b]) + S, T)   # tokens that any row sees
        last = max(last, 0)
        for i, pg in enumerate(row):
            lo = min(max(last - i * page, 0), page)
            raw(a["kc"])[pg, lo:] = 0x7f
            raw(a["vc"])[pg, lo:] = 0xff
            g = -(-lo // group)
            a["ks"][pg, g:] = math.nan
            a["vs"][pg, g:] = math.inf
    o2, lse2, _ = call(dsa, a)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert any(not torch.equal(raw(a[n]), raw(clean[n])) for n in ("kc", "vc"))


@gpu
@pytest.mark.parametrize("case", [ATTN[8], ATTN[9], ATTN[12], ATTN[13]])
@pytest.mark.parametrize("which", ["kc", "vc"])
def test_attention_nan_reaches_only_rows_that_see_it(dsa, case, which):
    a = attn_inputs(case, 4)
    b, S = 0, a["q"].shape[0]
    j = int(a["q_pos"][0]) + S // 2           # half of the rows see it
    page = a["kc"].shape[1]
    raw(a[which])[int(a["table"][b, j // page]), j % page, :, 3] = 0x7f
    o, lse, _ = call(dsa, a)
    o = o.cpu()
    clean = dict(a, **{which: a[which].clone()})
    raw(clean[which])[int(a["table"][b, j // page]), j % page, :, 3] = 0
    r, T = reference(clean)
    pos = int(a["q_pos"][0])
    for s in range(S):
        for hk in range(a["kc"].shape[2]):
            G = a["q"].shape[2] // a["kc"].shape[2]
            hs = slice(hk * G, hk * G + G)
            sees = j in row_keys(a["ids"], b, s, hk, pos + s, a["block"],
                                 a["local"], T)
            got = torch.isnan(o[s, b, hs].float())
            if which == "kc":
                assert bool(got.all()) == sees
                assert bool(torch.isnan(lse[s, b, hs]).all()) == sees
            else:
                assert bool(got[:, 3].all()) == sees
                assert not bool(got[:, :3].any())
            if sees:  # compared below as what a clean cache gives
                o[s, b, hs] = r["o"][s, b, hs].to(BF)
                lse[s, b, hs] = r["lse"][s, b, hs].float().cuda()
    check_attn(r, o, lse, T)


@gpu
@pytest.mark.parametrize("case", [ATTN[1], ATTN[3], ATTN[9], ATTN[12]])
def test_attention_scales_far_apart(dsa, case):
    """Groups whose scales differ by up to 2^60, a head whose values are all
    zeros, queries of any size."""
    a = attn_inputs(case, 6)
    g = torch.Generator().manual_seed(2)
    a["vs"] = 2.0 ** torch.randint(-30, 31, a["vs"].shape, generator=g).float()
    raw(a["vc"])[:, :a["group"]] = 0
    a["vs"][:, 0] = 2.0 ** -40
    a["ks"] = 2.0 ** torch.randint(-12, -6, a["ks"].shape, generator=g).float()
    a["q"] = (a["q"].float() * 2.0 ** torch.randint(
        -3, 4, a["q"].shape[:3] + (1,), generator=g)).to(BF)
    o, lse, _ = call(dsa, a)
    r, T = reference(a)
    # per row: the largest product of a weight and a scale
    r["w_top"] = w_top(a, T)
    check_attn(r, o, lse, T)


def w_top(a, T):
    S, B, H, D = a["q"].shape
    Hk = a["kc"].shape[2]
    out = torch.zeros((S, B, H, 1)).double()
    k = dense(a["kc"], a["ks"], a["table"], a["group"])
    one = torch.ones(a["kc"].shape[:3] + (1,))
    sv = dense(one, a["vs"], a["table"], a["group"])
    for b in range(B):
        for s in range(S):
            for h in range(H):
                hk = h // (H // Hk)
                js = row_keys(a["ids"], b, s, hk, int(a["q_pos"][b]) + s,
                              a["block"], a["local"], T)
                if js:
                    x = a["scale"] * k[b][js, hk] @ a["q"][s, b, h].double()
                    w = torch.softmax(x, 0) * sv[b][js, hk, 0]
                    out[s, b, h] = w.max()
    return out


@gpu
def test_attention_reports_bad_ids_and_pages(dsa):
    a = attn_inputs(ATTN[1], 7)
    a["q_pos"][:] = 300
    good = a["ids"].clone()
    a["ids"][0, 0, 0, 0] = 6
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 6
    a["ids"][0, 0, 0, 0] = -1
    r, T = reference(a)
    check_attn(r, o, lse, T)
    a["ids"] = good
    a["ids"][:] = -1
    a["ids"][2, 0, 1, 0] = 1
    page = int(a["table"][2, 1])
    a["table"][2, 1] = a["kc"].shape[0]
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 6
    a["table"][2, 1] = page
    a["ids"][2, 0, 1, 0] = -1
    r, T = reference(a)
    check_attn(r, o, lse, T)


@gpu
@pytest.mark.parametrize("case", [ATTN[0], ATTN[6], ATTN[9], ATTN[13], ATTN[16]])
def test_attention_skips_bad_pages(dsa, case):
    """A page that the table names wrongly is left out and reported; pages
    behind a row's position are not looked at."""
    a = attn_inputs(case, 7)
    page, S = a["kc"].shape[1], a["q"].shape[0]
    T = page * a["table"].shape[1]
    a["q_pos"][:] = T - S - 1 - page // 2
    a["ids"] = None
    a["local"] = T // a["block"]
    if case[7] != 99:                        # the selection's kernel
        n = -(-T // a["block"])
        a["ids"] = torch.arange(n).expand(a["q"].shape[1], S, n).contiguous(
        ).to(torch.int32)
        a["local"] = 1
    good = a["table"].clone()
    a["table"][0, -1] = -7                   # behind the rows
    o, lse, ws = call(dsa, a)
    seen = int(a["q_pos"][0]) + S - 1 >= T - page
    assert dsa.dsa_indexer_check(ws) == (6 if seen else 0)
    a["table"] = good.clone()
    a["table"][0, 0] = a["kc"].shape[0]
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 6
    # sequence 0 as if its first page's scores were -inf
    k, v = (torch.stack(dense(c, s, good, a["group"]), 1)
            for c, s in ((a["kc"], a["ks"]), (a["vc"], a["vs"])))
    H, Hk = a["q"].shape[2], a["kc"].shape[2]
    for s in (0, S - 1):
        for h in (0, H - 1):
            hk = h // (H // Hk)
            js = slice(page, int(a["q_pos"][0]) + s + 1)
            x = a["scale"] * k[js, 0, hk] @ a["q"][s, 0, h].double()
            p = torch.softmax(x, 0)
            want = p @ v[js, 0, hk]
            tol = (2.0 ** -10 * (p @ v[js, 0, hk].abs())
                   + 2.0 ** -8 * want.abs() + T * 2.0 ** -27)
            got = o[s, 0, h].double().cpu()
            assert bool(((got - want).abs() <= tol).all())


@gpu
@pytest.mark.parametrize("case", [ATTN[1], ATTN[6], ATTN[9], ATTN[12], ATTN[16]])
def test_attention_of_queries_that_are_not_finite(dsa, case):
    """A NaN or an infinity in a query stays in its row; queries of zeros and
    of the smallest and largest sizes are like others."""
    a = attn_inputs(case, 11)
    H = a["q"].shape[2]
    rows = [(0, 0, 0), (a["q"].shape[0] - 1, 0, H - 1)]
    a["q"][rows[0]][5] = math.nan
    a["q"][rows[1]][7] = math.inf
    a["q"][0, -1, 0] = 0
    a["q"][0, -1, 1 % H] *= 2.0 ** -120
    o, lse, _ = call(dsa, a)
    clean = dict(a, q=a["q"].clone())
    for r in rows:
        clean["q"][r] = 0
    r, T = reference(clean)
    o, lse = o.cpu(), lse.cpu()
    for x in rows:
        assert bool(torch.isnan(o[x]).all()) == (float(r["lse"][x]) > -math.inf)
        o[x], lse[x] = r["o"][x].to(BF), r["lse"][x].float()
    check_attn(r, o, lse, T)


@gpu
@pytest.mark.parametrize("case", [ATTN[1], ATTN[6], ATTN[12]])
def test_streams_and_graphs(dsa, case):
    """Calls on a stream of their own, and two captured graphs that share a
    workspace, replayed in turn with new inputs."""
    a, b = attn_inputs(case, 8), attn_inputs(case, 9)
    want = [call(dsa, x)[:2] for x in (a, b)]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(dsa, a, stream=st)
    st.synchronize()
    assert torch.equal(got[0], want[0][0])
    dev = {n: (t.cuda() if isinstance(t, torch.Tensor) else t)
           for n, t in a.items()}
    ws = got[2]
    outs, graphs = [], []
    for _ in range(2):
        o, lse = torch.zeros_like(want[0][0]), torch.zeros_like(want[0][1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(dsa, dev, out_o=o, out_lse=lse, workspace=ws)
        outs.append((o, lse))
        graphs.append(graph)
    for i in range(4):
        src = (a, b)[i % 2]
        for n, t in dev.items():
            if isinstance(t, torch.Tensor):
                t.copy_(src[n])
        graphs[i // 2].replay()
        torch.cuda.synchronize()
        o, lse = outs[i // 2]
        assert torch.equal(o, want[i % 2][0])
        assert torch.equal(lse, want[i % 2][1])
    assert dsa.dsa_indexer_check(ws) == 0


@gpu
@pytest.mark.parametrize("case", [
    # S, B, H, Hk, D, block, topk, local, shared, page, group, pages
    (40, 42, 8, 4, 64, 16, 2, 1, False, 32, 16, 3),
    (33, 80, 6, 2, 128, 32, 0, 99, True, 32, 32, 3),
    (5, 200, 17, 1, 128, 64, 2, 1, True, 64, 64, 2),
    (7, 170, 33, 1, 64, 128, 0, 99, True, 128, 128, 1),
])
def test_attention_of_many_tiles(dsa, case):
    """Enough tiles that none is cut into parts."""
    a = attn_inputs(case, 10)
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(a)
    check_attn(r, o, lse, T)


@gpu
@pytest.mark.parametrize("case", [
    # block lists that leave the ring of a single token one stage, and those of
    # a tile with every block that there may be
    (1, 2, 4, 1, 128, 16, 9000, 3, True, 1024, 128, 256),
    (1, 1, 3, 1, 64, 16, 16000, 1, True, 4096, 64, 64),
    (33, 1, 2, 1, 128, 16, 700, 2, True, 1024, 128, 256),
    (33, 1, 2, 1, 64, 16, 700, 2, True, 1024, 128, 256),
])
def test_attention_of_the_longest_lists(dsa, case):
    a = attn_inputs(case, 11)
    a["q_pos"][0] = case[9] * case[11] - case[0]
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(a)
    r["w_top"] = w_top(a, T)
    check_attn(r, o, lse, T)


@gpu
@pytest.mark.parametrize("S,H,D", [(3, 4, 64), (2, 8, 128), (2, 24, 64)])
def test_attention_of_the_longest_cache(dsa, S, H, D):
    """All of 2^21 keys: as many steps as an item can have.  (The last case
    takes the kernel for many rows.)"""
    page, group, block = 4096, 128, 128
    T = 1 << 21
    g = torch.Generator(device="cuda").manual_seed(D + H)
    kc, vc = ((torch.randn((T // page, page, 1, D), generator=g, device="cuda")
               * 100).clamp(-448, 448).to(E4M3) for _ in "kv")
    ks, vs = (2.0 ** torch.randint(-9, -4, (T // page, page // group, 1),
                                   generator=g, device="cuda").float()
              for _ in "kv")
    table = torch.randperm(T // page, generator=g, device="cuda")
    table = table.to(torch.int32)[None]
    q = torch.randn((S, 1, H, D), generator=g, device="cuda").to(BF)
    q_pos = torch.tensor([T - S], dtype=torch.int32, device="cuda")
    o, lse, ws = dsa.dsa_block_attn_paged_q8_fwd(
        q, kc, vc, ks, vs, table, None, block, 0.11, q_pos=q_pos,
        local_blocks=T // block)
    assert dsa.dsa_indexer_check(ws) == 0
    order = table[0].long()
    k, v = ((c.double() * s.double().repeat_interleave(group, 1)[..., None])
            [order].view(T, D) for c, s in ((kc, ks), (vc, vs)))
    scale_of = vs.double().repeat_interleave(group, 1)[order].view(T)
    r = {n: torch.zeros((S, 1, H, D), dtype=torch.float64) for n in ("o", "A_o")}
    r["lse"], r["X"] = (torch.zeros((S, 1, H), dtype=torch.float64)
                        for _ in "ab")
    r["w_top"] = torch.zeros((S, 1, H, 1), dtype=torch.float64)
    for s in range(S):
        n = T - S + s + 1
        x = 0.11 * q[s, 0].double() @ k[:n].T
        z = torch.logsumexp(x, 1)
        w = torch.exp(x - z[:, None])
        r["o"][s, 0], r["lse"][s, 0] = (w @ v[:n]).cpu(), z.cpu()
        r["A_o"][s, 0] = (w @ v[:n].abs()).cpu()
        r["X"][s, 0] = (0.11 * q[s, 0].double().abs()
                        @ k[:n].abs().T).amax(1).cpu()
        r["w_top"][s, 0, :, 0] = (w * scale_of[:n]).amax(1).cpu()
    check_attn(r, o, lse, T)


# ---- together, streams, threads ---------------------------------------------------

@gpu
def test_a_layer_served(dsa):
    """A prompt in two chunks and single tokens: append, read back, block means,
    selection, attention.  Each step's output is the definition's on what the
    cache holds after it, and the cache is that of one append of all tokens."""
    S, B, H, Hk, D, block, page = 75, 2, 8, 2, 64, 16, 32
    pages = 3
    g = torch.Generator().manual_seed(12)
    qkv = torch.randn((S, B, H + 2 * Hk, D), generator=g).to(BF).cuda()
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    f = inv(D).cuda()
    table = torch.randperm(B * pages, generator=g).to(torch.int32).view(B, pages)
    table = table.cuda()
    cache = [t.cuda() for t in make_cache(B * pages, page, Hk, D, 16, 1)]
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    steps = [(0, 40), (40, 71)] + [(s, s + 1) for s in range(71, S)]
    for s0, s1 in steps:
        x = qkv[s0:s1]
        start = torch.full((B,), s0, dtype=torch.int32, device="cuda")
        q, _ = dsa.dsa_paged_append_q8(
            x[:, :, H:H + Hk], x[:, :, H + Hk:], *cache, table, start,
            inv_freq=f, wk=w, q=x[:, :, :H], wq=w, workspace=status)
        k, v, _ = dsa.dsa_paged_read_q8(*cache, table, s1, workspace=status)
        n = s1 // block
        means = k[:n * block, :, 0].float().view(n, block, B, D).mean(1).to(BF)
        wi = torch.full((s1 - s0, B, H), 1.0 / H, device="cuda")
        _, ids = dsa.v4_lighting_indexer(q, means, wi, block, 2, q_pos=start)
        o, lse, ws = dsa.dsa_block_attn_paged_q8_fwd(
            q, *cache, table, ids, block, 0.125, q_pos=start, local_blocks=1)
        assert dsa.dsa_indexer_check(ws) == 0
        r = block_attn_ref(q.cpu(), k.cpu(), v.cpu(), ids.cpu(), block, 1,
                           0.125, q_pos=start.cpu())
        check_attn(r, o, lse, s1)
    assert dsa.dsa_indexer_check(status) == 0
    once = [t.cuda() for t in make_cache(B * pages, page, Hk, D, 16, 1)]
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    dsa.dsa_paged_append_q8(qkv[:, :, H:H + Hk], qkv[:, :, H + Hk:], *once,
                            table, zero, inv_freq=f, wk=w)
    a = dsa.dsa_paged_read_q8(*cache, table, S)
    b = dsa.dsa_paged_read_q8(*once, table, S)
    for i in (0, 1):
        # (codes that were subnormal on the way are a step apart at most)
        step = cache[2 + i].amax() * 2.0 ** -9
        assert float((a[i].float() - b[i].float()).abs().max()) <= float(step)


@gpu
@pytest.mark.parametrize("S", [1, 20])
def test_a_step_captured(dsa, S):
    """Append, attention over all keys and read back in one graph, replayed as
    the sequences grow; a sequence that is not served keeps its cache."""
    B, H, Hk, D, page, group, pages = 3, 8, 2, 64, 64, 32, 4
    g = torch.Generator().manual_seed(S)
    cache = [t.cuda() for t in make_cache(B * pages, page, Hk, D, group, 4)]
    eager = [t.clone() for t in cache]
    table = torch.randperm(B * pages, generator=g).to(torch.int32)
    table = table.view(B, pages).cuda()
    f = inv(D).cuda()
    x = torch.zeros((S, B, H + 2 * Hk, D), dtype=BF, device="cuda")
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    count = torch.zeros(B, dtype=torch.int32, device="cuda")
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    size = dsa.dsa_block_attn_q8_workspace_size(S, B, H, Hk, D, page * pages,
                                                16, 0, page * pages // 16)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def step(c):
        q, _ = dsa.dsa_paged_append_q8(
            x[:, :, H:H + Hk], x[:, :, H + Hk:], *c, table, start, count,
            inv_freq=f, q=x[:, :, :H], workspace=status)
        o, lse, _ = dsa.dsa_block_attn_paged_q8_fwd(
            q, *c, table, None, 16, 0.125, q_pos=start,
            local_blocks=page * pages // 16, workspace=ws)
        k, v, _ = dsa.dsa_paged_read_q8(*c, table, page * pages, length=count,
                                        workspace=status)
        return q, o, lse, k, v

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):        # (appends nothing: counts are zero)
        step([t.clone() for t in cache])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(cache)
    at = [0, 37, 100]
    untouched = [raw(t)[table[1].long()].clone() if t.dtype is E4M3
                 else t[table[1].long()].clone() for t in cache]
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=g).to(BF))
        n = [S, 0, S - S // 3]
        start.copy_(torch.tensor(at, dtype=torch.int32))
        count.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        want = step(eager)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for a, b in zip(cache, eager):
            assert torch.equal(raw(a), raw(b))
        at = [p + m for p, m in zip(at, n)]
    for t, was in zip(cache, untouched):
        now = t[table[1].long()] if t.dtype is not E4M3 else \
            raw(t)[table[1].long()]
        assert torch.equal(now, was)
    assert dsa.dsa_indexer_check(status) == 0
    assert dsa.dsa_indexer_check(ws) == 0


@gpu
def test_example_serves_from_8_bits(dsa):
    """The example's layer from either cache: the outputs differ by the
    rounding of keys and values, 2^-4 each at most where one selects the same
    blocks."""
    import importlib.util
    import os
    import sys
    path = os.path.join(os.path.dirname(os.path.dirname(
        os.path.abspath(__file__))), "examples", "block_sparse_layer.py")
    spec = importlib.util.spec_from_file_location("block_sparse_layer_q8", path)
    m = importlib.util.module_from_spec(spec)
    sys.modules["block_sparse_layer_q8"] = m
    spec.loader.exec_module(m)
    # every block is local: no selection that a rounding could change
    layer = m.Layer(hidden=64, local=4, topk=1)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((150, 2, 64), generator=g, device="cuda").to(BF)
    a = layer.serve(x, prompt=140).float()
    b = layer.serve(x, prompt=140, bits=8).float()
    assert bool(torch.isfinite(b).all())
    # (norms: a softmax's output moves by at most the values' 2^-4 and twice
    # the scores' 2^-4 |q| |k| scale < 2^-4 * 12 of the values' spread, most of
    # which averages out; a quarter would be another layer)
    assert float((a - b).norm() / a.norm()) < 0.25


def q8_calls(dsa):
    """name -> call(stream): what is compared."""
    a = attn_inputs(ATTN[1], 8)
    dev = {n: (t.cuda() if isinstance(t, torch.Tensor) else t)
           for n, t in a.items()}
    many = {n: (t.cuda() if isinstance(t, torch.Tensor) else t)
            for n, t in attn_inputs(ATTN[12], 8).items()}
    k = torch.randn((37, 3, 2, 128), device="cuda").to(BF)
    start = torch.tensor([0, 70, 300], dtype=torch.int32, device="cuda")
    bad = torch.full_like(dev["table"], 10 ** 6)
    f = inv(128).cuda()
    cache = (dev["kc"], dev["vc"], dev["ks"], dev["vs"])
    copies = tuple(t.clone() for t in cache)
    return {
        "append": lambda st: dsa.dsa_paged_append_q8(
            k, k, *copies, dev["table"], start, inv_freq=f, q=k,
            stream=st)[:1],
        "append, bad page": lambda st: (dsa.dsa_paged_append_q8(
            k, k, *copies, bad, start, stream=st)[1][:4],),
        "read": lambda st: dsa.dsa_paged_read_q8(*cache, dev["table"], 99,
                                                 stream=st)[:2],
        "one token": lambda st: call(dsa, dev, stream=st)[:2],
        "chunk": lambda st: call(dsa, many, stream=st)[:2],
    }


@gpu
def test_given_stream(dsa):
    """Calls on a stream of their own, while blocks of their outputs' and
    workspaces' sizes are freed with work queued on the current one."""
    side = torch.cuda.Stream()
    for name, fn in q8_calls(dsa).items():
        want = [t.clone() for t in fn(None)]
        torch.cuda.synchronize()
        sizes = [t.numel() * t.element_size() for t in want]
        held = [torch.empty(n, dtype=torch.uint8, device="cuda")
                for n in sizes + [256, 1 << 12, 1 << 16, 6 << 20] for _ in "ab"]
        torch.cuda.synchronize()
        torch.cuda._sleep(60_000_000)      # some 30 ms
        for t in held:
            t.fill_(255)
        del held, t
        got = fn(side)
        side.synchronize()
        with torch.cuda.stream(side):
            early = [t.clone().cpu() for t in got]
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, early):
            assert torch.equal(a, b), name
            assert torch.equal(a.cpu(), c), name


@gpu
def test_two_threads(dsa):
    """Two threads with streams and workspaces of their own at once."""
    import threading
    calls = q8_calls(dsa)
    want = {n: [t.clone() for t in fn(None)] for n, fn in calls.items()
            if not n.startswith("append")}
    torch.cuda.synchronize()
    errors = []

    def work(seed):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(30):
                    for n in want:
                        for a, b in zip(calls[n](None), want[n]):
                            if not torch.equal(a, b):
                                errors.append(n)
            st.synchronize()
        except Exception as e:  # pragma: no cover
            errors.append(repr(e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors


@gpu
def test_wrong_tensors_are_refused(dsa):
    a = attn_inputs(ATTN[1], 8)
    dev = {n: (t.cuda() if isinstance(t, torch.Tensor) else t)
           for n, t in a.items()}

    def refused(err, match, **over):
        with pytest.raises(err, match=match):
            call(dsa, dict(dev, **over))
    refused(TypeError, "q must be", q=dev["q"].float())
    refused(ValueError, "contiguous", q=dev["q"].transpose(0, 2))
    refused(TypeError, "k_cache must be", kc=raw(dev["kc"]))
    refused(ValueError, "v_cache shape", vc=dev["vc"][:-1])
    refused(ValueError, "k_scale shape", ks=dev["ks"][:-1])
    refused(TypeError, "v_scale must be", vs=dev["vs"].double())
    refused(ValueError, "do not divide", ks=dev["ks"].repeat(1, 3, 1))
    refused(ValueError, "page_table is for", table=dev["table"][:2])
    refused(ValueError, "blocks shape", ids=dev["ids"][:, :, :1])
    refused(ValueError, "q_pos shape", q_pos=dev["q_pos"][:2])
    k = torch.zeros((3, 3, 2, 128), dtype=BF, device="cuda")
    cache = (dev["kc"], dev["vc"], dev["ks"], dev["vs"], dev["table"])
    start = torch.zeros(3, dtype=torch.int32, device="cuda")
    for over, err in ((dict(start=start[:2]), ValueError),
                      (dict(start=start.long()), TypeError),
                      (dict(count=start.float()), TypeError),
                      (dict(k=k[:, :2]), ValueError),
                      (dict(k=k.float()), TypeError),
                      (dict(v=k[..., :64]), ValueError),
                      (dict(wk=start.float()), ValueError),
                      (dict(q=k.half()), TypeError)):
        kw = dict(dict(k=k, v=k, start=start), **over)
        with pytest.raises(err):
            dsa.dsa_paged_append_q8(
                kw.pop("k"), kw.pop("v"), *cache, kw.pop("start"), **kw)
    with pytest.raises(TypeError):
        dsa.dsa_paged_read_q8(*cache, 5, first=start.long())
    with pytest.raises(ValueError):
        dsa.dsa_paged_read_q8(*cache, 5, out_k=k)


# ---- references and refusals (no GPU) --------------------------------------------

def test_reference_e4m3_against_torch():
    x = torch.cat([torch.randn(20000) * 100, torch.randn(20000) * 0.01,
                   torch.arange(0, 500, 0.25), torch.arange(0, 0.2, 2.0 ** -11)])
    x = torch.cat([x, -x]).clamp(-448, 448)
    assert torch.equal(to_e4m3(x), x.to(E4M3).double())


def test_reference_scale():
    from tests.cache_q8_ref import exp_for
    for e in (-20, -3, 0, 7):
        top = 448 * 2.0 ** e
        assert exp_for(top) == e
        assert exp_for(math.nextafter(top, 0)) == e
        assert exp_for(math.nextafter(top, math.inf)) == e + 1
    assert exp_for(0.0) == -40 and exp_for(1e30) == 40


def test_calls_refuse(dsa):
    x = torch.zeros((2, 1, 2, 64), dtype=BF)
    c = torch.zeros((2, 16, 2, 64), dtype=torch.uint8).view(E4M3)
    s = torch.ones((2, 1, 2))
    t = torch.zeros((1, 2), dtype=torch.int32)
    p = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dsa.dsa_paged_append_q8(x, x, c, c, s, s, t, p)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dsa.dsa_paged_read_q8(c, c, s, s, t, 4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dsa.dsa_block_attn_paged_q8_fwd(x, c, c, s, s, t, None, 16, 0.1,
                                        local_blocks=1)


FAKE = 1 << 20  # aligned, never read: every case fails before its use
CACHE = [
    (dict(kc=None), 1), (dict(vc=None), 1), (dict(ks=None), 1),
    (dict(vs=None), 1), (dict(table=None), 1), (dict(group=0), 1),
    (dict(group=8), 2), (dict(group=48, page=48), 2), (dict(page=24), 2),
    (dict(pages=0), 1), (dict(page=0), 1), (dict(maxp=0), 1),
    (dict(D=72), 2), (dict(D=288), 2), (dict(kc=FAKE + 8), 1),
    (dict(ks=FAKE + 2), 1), (dict(table=FAKE + 1), 1),
    (dict(maxp=1 << 27), 2), (dict(ws=None), 3), (dict(wsb=255), 3),
    (dict(ws=FAKE + 16), 1), (dict(Hk=0), 1),
]


@pytest.mark.parametrize("over,code", CACHE + [
    (dict(k=None), 1), (dict(v=None), 1), (dict(start=None), 1),
    (dict(start=FAKE + 2), 1), (dict(count=FAKE + 2), 1), (dict(S=0), 1),
    (dict(q=FAKE, H=2), 1), (dict(R=3), 1), (dict(R=4), 1),
    (dict(eps=math.nan), 1), (dict(D=256, group=128, page=128), 2),
    (dict(k=FAKE + 1), 1), (dict(B=1 << 20, S=1 << 12), 2),
])
def test_append_refuses(dsa, over, code):
    a = dict(k=FAKE, k_st=None, v=FAKE, v_st=None, q=None, q_st=None, S=1,
             B=1, H=0, Hk=1, D=64, kc=FAKE, vc=FAKE, cs=None, ks=FAKE, vs=FAKE,
             group=16, pages=2, page=16, table=FAKE, maxp=2, start=FAKE,
             count=None, wq=None, wk=None, eps=1e-6, inv=None, r0=0, R=0,
             inter=0, m=1.0, oq=None, ws=FAKE, wsb=256, st=None)
    a.update(over)
    assert dsa.load_library().dsa_paged_append_q8(*a.values()) == code


@pytest.mark.parametrize("over,code", CACHE + [
    (dict(ok=None, ov=None), 1), (dict(T=0), 1), (dict(B=0), 1),
    (dict(ok=FAKE + 8), 1), (dict(first=FAKE + 1), 1),
    (dict(T=1 << 20, B=1 << 12), 2),
])
def test_read_refuses(dsa, over, code):
    a = dict(kc=FAKE, vc=FAKE, cs=None, ks=FAKE, vs=FAKE, group=16, pages=2,
             page=16, table=FAKE, maxp=2, T=4, B=1, Hk=1, D=64, first=None,
             length=None, ok=FAKE, ov=FAKE, ws=FAKE, wsb=256, st=None)
    a.update(over)
    assert dsa.load_library().dsa_paged_read_q8(*a.values()) == code


@pytest.mark.parametrize("over,code", CACHE[:-1] + [
    (dict(q=None), 1), (dict(o=None), 1), (dict(lse=None), 1),
    (dict(Hk=0), 1), (dict(H=3, Hk=2), 1), (dict(S=0), 1),
    (dict(topk=2, blocks=None), 1), (dict(local=0), 1), (dict(local=-1), 1),
    (dict(sel=2, Hk=1), 1), (dict(block=48), 2), (dict(block=32), 2),
    (dict(D=96), 2), (dict(H=65), 2), (dict(scale=0.0), 1),
    (dict(scale=math.nan), 1), (dict(o=FAKE + 8), 1), (dict(q=FAKE + 8), 1),
    (dict(local=16385), 2), (dict(maxp=1 << 18), 2),
])
def test_attention_refuses(dsa, over, code):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, cs=None, ks=FAKE, vs=FAKE, group=16,
             pages=2, page=16, table=FAKE, maxp=2, S=1, B=1, H=1, Hk=1, D=64,
             blocks=None, sel=1, topk=0, block=16, local=1, q_pos=None,
             scale=0.1, o=FAKE, lse=FAKE, ws=FAKE, wsb=256, st=None)
    a.update(over)
    if "wsb" not in over and over.get("ws", 1):
        a["wsb"] = 1 << 40
    got = dsa.load_library().dsa_block_attn_paged_q8_fwd(*a.values())
    assert got == code


def test_strides_are_checked(dsa):
    import ctypes
    lib = dsa.load_library()
    for bad in ([0, 64, 64], [2048, 0, 64], [2048, 128, 8], [-16, 128, 64],
                [1 << 41, 128, 64], [2048, 72, 64]):
        cs = (ctypes.c_int64 * 6)(*(bad + [2048, 128, 64]))
        rc = lib.dsa_paged_read_q8(
            FAKE, FAKE, cs, FAKE, FAKE, 16, 2, 16, FAKE, 2, 4, 1, 2, 64, None,
            None, FAKE, FAKE, FAKE, 256, None)
        assert rc == 1, bad
    assert dsa.dsa_block_attn_q8_workspace_size(1, 1, 3, 2, 64, 64, 16, 1) == 0
    assert dsa.dsa_block_attn_q8_workspace_size(1, 1, 4, 2, 64, 64, 16, 1) >= 256
