"""The 8-bit cache at the ends of its ranges: queries of any size, keys that
decide a long row, appends of every width, rows that are not finite.

Tolerances are those of tests/test_cache_q8.py (their sums are written down
there)."""
from __future__ import annotations

import pytest
import torch

from tests.block_ref import norm_rope_ref, row_keys
from tests.cache_q8_ref import E4M3, dense
from tests.test_cache_q8 import (ATTN, BF, EPS, attn_inputs, call,
                                 check_append, check_attn, dsa, inv,
                                 make_cache, raw, reference, weights,
                                 test_append as append_as,
                                 test_append_of_unaligned_rows as
                                 append_unaligned_as)  # noqa: F401

gpu = pytest.mark.gpu

# of both attention kernels: over a selection and over all keys
KERNELS = [ATTN[1], ATTN[6], ATTN[9], ATTN[21], ATTN[5], ATTN[12], ATTN[13]]


@gpu
@pytest.mark.parametrize("power", [108, 112, 116, 120])
@pytest.mark.parametrize("case", KERNELS)
def test_large_queries_with_a_small_scale(dsa, case, power):
    """The scale brings the scores back to ordinary ones: the same softmax as
    that of ordinary queries, power for power.  (Powers of two: exact.)"""
    a = attn_inputs(case, 21)
    a["scale"] = 0.109375               # exact in fp32 after the power, too
    want = call(dsa, a)
    big = dict(a, q=(a["q"].float() * 2.0 ** power).to(BF),
               scale=a["scale"] * 2.0 ** -power)
    assert bool(torch.isfinite(big["q"].float()).all())
    o, lse, ws = call(dsa, big)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(big)
    check_attn(r, o, lse, T)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@gpu
@pytest.mark.parametrize("power", [108, 112, 116, 120])
@pytest.mark.parametrize("case", [c for c in KERNELS if c[0] < 33 and
                                  c[2] // c[3] <= 16])
def test_rows_of_large_queries(dsa, case, power):
    """Large queries among ordinary ones: the row's largest score takes all of
    its weight, and a row of one key gives that key's value."""
    a = attn_inputs(case, 22)
    a["q_pos"][0] = 0
    a["q"][0, 0] = (a["q"][0, 0].float() * 2.0 ** power).to(BF)
    a["q"][-1, -1, 0] = (a["q"][-1, -1, 0].float() * 2.0 ** power).to(BF)
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(a)
    assert float(r["lse"][0, 0].abs().min()) > 2.0 ** (power - 20)
    check_attn(r, o, lse, T)


@gpu
@pytest.mark.parametrize("power", [20, 24, 26, 28, 31, 35, 40, 64, 100, 120])
@pytest.mark.parametrize("case", KERNELS)
def test_large_scores_of_one_key(dsa, case, power):
    """Rows of one key, with scores of either sign and any size."""
    a = attn_inputs(case, 23)
    a["q_pos"][0] = 0
    a["q"][0, 0] = (a["q"][0, 0].float() * 2.0 ** power).to(BF)
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(a)
    row = r["lse"][0, 0]
    assert row.numel() < 4 or bool((row < 0).any()) and bool((row > 0).any())
    check_attn(r, o, lse, T)
    assert bool((o[0, 0].double().cpu() - r["o"][0, 0]).abs().max() <= 2.0 ** -8
                * r["o"][0, 0].abs().max())


@gpu
@pytest.mark.parametrize("power", [64, 112, 120])
@pytest.mark.parametrize("case", [ATTN[5], ATTN[12], ATTN[13]])
def test_rows_of_large_queries_in_tiles(dsa, case, power):
    """(As above, of the kernel for many rows.)"""
    a = attn_inputs(case, 22)
    a["q"][0, 0] = (a["q"][0, 0].float() * 2.0 ** power).to(BF)
    a["q"][-1, -1, 0] = (a["q"][-1, -1, 0].float() * 2.0 ** power).to(BF)
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(a)
    check_attn(r, o, lse, T)


def long_cache(S, B, H, Hk, D, T, page, group, seed):
    """Sequences that share one long prefix, in every page of a cache."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    kc, vc = ((torch.randn((T // page, page, Hk, D), generator=g, device="cuda")
               * 100).clamp(-448, 448).to(E4M3) for _ in "kv")
    ks, vs = (2.0 ** torch.randint(-9, -5, (T // page, page // group, Hk),
                                   generator=g, device="cuda").float()
              for _ in "kv")
    table = torch.randperm(T // page, generator=g, device="cuda").to(torch.int32)
    q = torch.randn((S, B, H, D), generator=g, device="cuda").to(BF)
    pos = torch.full((B,), T - S - 7, dtype=torch.int32, device="cuda")
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table.repeat(B, 1),
                q_pos=pos)


def attend(dsa, a, ids=None, block=128, **over):
    a = dict(a, **over)
    T = a["table"].shape[1] * a["kc"].shape[1]
    o, lse, ws = dsa.dsa_block_attn_paged_q8_fwd(
        a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], ids, block, 0.11,
        q_pos=a["q_pos"], local_blocks=1 if ids is not None else T // block)
    assert dsa.dsa_indexer_check(ws) == 0      # no wait expired
    return o, lse


@gpu
@pytest.mark.parametrize("S,B,H,Hk,D,T", [
    (1, 40, 32, 4, 128, 1 << 17),    # more than one item a CTA
    (1, 3, 8, 1, 64, 1 << 17),
    (4, 40, 16, 4, 128, 1 << 17),    # rows that see different keys
    (2, 80, 32, 2, 64, 1 << 16),     # two row tiles
    (2, 3, 16, 1, 64, 1 << 21),      # the longest
    (40, 2, 8, 2, 128, 1 << 16),     # the kernel for many rows
    (40, 40, 40, 8, 64, 1 << 14),
])
def test_a_nan_in_a_long_cache(dsa, S, B, H, Hk, D, T):
    """A value that is not a number spoils its column of the rows that see it
    and nothing else, a key the rows that see it; the call ends in time."""
    page, group = 2048, 64
    a = long_cache(S, B, H, Hk, D, T, page, group, 31)
    o, lse = attend(dsa, a)
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
    # sum of weights times magnitudes: the same softmax over |v|
    A, _ = attend(dsa, a, vc=(raw(a["vc"]) & 0x7f).view(E4M3))
    tol = (2 * (2.0 ** -11 + 2.0 ** -12) * A.double() * (1 + 2.0 ** -7)
           + 2 * 2.0 ** -8 * o.double().abs() + T * 2.0 ** -21
           * float(a["vs"].max()))
    late = T - S - 7 + S // 2             # seen by the rows from S // 2 on
    G = H // Hk
    for j, s0 in ((5, 0), (late, S // 2)):
        for which in ("vc", "kc"):
            c = raw(a[which]).clone()
            c[int(a["table"][0, j // page]), j % page, Hk - 1, 3] = 0x7f
            o2, lse2 = attend(dsa, a, **{which: c.view(E4M3)})
            sees = torch.zeros((S, B, H), dtype=torch.bool, device="cuda")
            sees[s0:, :, H - G:] = True
            if which == "vc":
                bad = torch.zeros_like(o, dtype=torch.bool)
                bad[..., 3] = sees
                bad_l = torch.zeros_like(sees)
            else:
                bad, bad_l = sees[..., None].expand_as(o), sees
            assert torch.equal(torch.isnan(o2), bad)
            assert torch.equal(torch.isnan(lse2), bad_l)
            err = (o2.double() - o.double()).abs()
            assert bool((err <= tol)[~bad].all())
            d = (lse2 - lse).abs()[~bad_l]
            assert bool((d <= 2.0 ** -14 * (1 + 0.11 * 448 * 2.0 ** -6 * 128 * 3)
                         ).all())


@gpu
@pytest.mark.parametrize("S,B,H,Hk,D", [(1, 70, 32, 4, 128), (3, 5, 8, 2, 64),
                                        (33, 3, 8, 2, 128)])
def test_a_nan_in_a_selection(dsa, S, B, H, Hk, D):
    """(As above, over selected blocks: some rows hold the block.)"""
    page, group, block, T = 2048, 64, 64, 1 << 16
    a = long_cache(S, B, H, Hk, D, T, page, group, 32)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(0, T // block - 4, (B, S, Hk, 30), generator=g,
                        device="cuda").to(torch.int32)
    ids[..., 3] = -1
    ids[:, S // 2:, Hk - 1, 3] = 0
    ids[ids == 0] = -1
    ids[:, S // 2:, Hk - 1, 3] = 0
    o, lse = attend(dsa, a, ids, block)
    A, _ = attend(dsa, a, ids, block, vc=(raw(a["vc"]) & 0x7f).view(E4M3))
    tol = (2 * (2.0 ** -11 + 2.0 ** -12) * A.double() * (1 + 2.0 ** -7)
           + 2 * 2.0 ** -8 * o.double().abs() + 2.0 ** -10 * float(a["vs"].max()))
    G = H // Hk
    sees = torch.zeros((S, B, H), dtype=torch.bool, device="cuda")
    sees[S // 2:, :, H - G:] = True
    for which in ("vc", "kc"):
        c = raw(a[which]).clone()
        c[int(a["table"][0, 0]), 9, Hk - 1, 3] = 0xff
        o2, lse2 = attend(dsa, a, ids, block, **{which: c.view(E4M3)})
        bad = torch.zeros_like(o, dtype=torch.bool)
        if which == "vc":
            bad[..., 3] = sees
        else:
            bad |= sees[..., None]
        assert torch.equal(torch.isnan(o2), bad)
        assert torch.equal(torch.isnan(lse2),
                           sees if which == "kc" else torch.zeros_like(sees))
        assert bool(((o2.double() - o.double()).abs() <= tol)[~bad].all())


# ---- appends of every width --------------------------------------------------

# head size, rotated part and its start, pairs of neighbours
WIDTHS = [(64, 64, 0, False), (48, 16, 16, True), (128, 64, 64, False),
          (96, 96, 0, True), (192, 64, 0, False), (256, 256, 0, True)]


@gpu
@pytest.mark.parametrize("S", [1, 2, 3, 4, 8, 9, 40, 150])
@pytest.mark.parametrize("width,group", [
    (w, n) for w in WIDTHS for n in (16, 32, 64, 128) if w[0] * n <= 16384])
def test_append_of_every_width(dsa, width, group, S):
    """As many new rows as a warp, two passes of a warp or a CTA take, in groups
    of every size, normed and rotated, beginning inside groups."""
    D, R, r0, inter = width
    append_as(dsa, (S, 4, 6, 2, D, R, r0, inter, 128, 4, group, S % 2 == 0,
                    S > 4), True)


@gpu
@pytest.mark.parametrize("S", [1, 2, 3, 100])
@pytest.mark.parametrize("D,R,group", [
    (64, 24, 128), (128, 36, 128), (112, 64, 16), (192, 64, 64), (256, 256, 16)])
def test_append_of_unaligned_rows_of_every_width(dsa, S, D, R, group):
    append_unaligned_as(dsa, S, D, R, group, True)


# ---- every key once -------------------------------------------------------------

@gpu
@pytest.mark.parametrize("S,H,D", [(3, 4, 64), (2, 8, 128), (2, 16, 64),
                                   (2, 24, 64), (40, 2, 128)])
def test_every_key_of_the_longest_cache_counts_once(dsa, S, H, D):
    """64 keys of 2^21 share the softmax, each with a value of its own: the
    first and the last ones that rows see, those at the borders of what a CTA
    takes, of pages and of groups.  A key that is lost or counts twice changes
    its column by all of it.  (The other scores are 0, these 40: 2^21 e^-40 of
    the weight is nothing.)"""
    page, group, block = 4096, 128, 128
    T = 1 << 21
    g = torch.Generator(device="cuda").manual_seed(D + H)
    kc, vc = (torch.zeros((T // page, page, 1, D), dtype=torch.uint8,
                          device="cuda") for _ in "kv")
    ones = torch.ones((T // page, page // group, 1), device="cuda")
    table = torch.randperm(T // page, generator=g, device="cuda")
    q = torch.ones((S, 1, H, D), dtype=BF, device="cuda")
    pos = T - S - 3
    # borders of the slices and of the parts that tiles are cut into
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    at = [0, 1, pos - 1, pos] + list(range(pos + 1, pos + S + 1))
    steps = (pos + S - 1) // 32 + 1
    share, more = steps // sms, steps % sms
    at += [32 * (c * share + c * more // sms) + d for c in range(1, sms)
           for d in (-1, 0)]
    for parts in (255, 2 * sms // max(1, S * H // 128), 152, 304):
        at += [64 * (T // 64 * c // parts) + d
               for c in torch.randint(1, parts, (24,)).tolist() for d in (-1, 0)]
    at += torch.randint(0, T, (64,)).tolist()
    at += [page * i + d for i in (1, 2, T // page - 1) for d in (-1, 0)]
    at += [group * i + d for i in (1, 77, T // group - 1) for d in (-1, 0)]
    at = sorted(set(at))
    one = int(torch.ones(1).to(E4M3).view(torch.uint8))
    for i in range(0, len(at), 64):
        js = torch.tensor(at[i:i + 64], device="cuda")
        pg, off = table[js // page], js % page
        kc[pg, off] = one
        vc[pg, off, 0, torch.arange(len(js), device="cuda")] = one
        o, lse, ws = dsa.dsa_block_attn_paged_q8_fwd(
            q, kc.view(E4M3), vc.view(E4M3), ones, ones,
            table.to(torch.int32)[None], None, block, 40.0 / D,
            q_pos=torch.tensor([pos], dtype=torch.int32, device="cuda"),
            local_blocks=T // block)
        assert dsa.dsa_indexer_check(ws) == 0
        kc[pg, off] = 0
        vc[pg, off] = 0
        for s in range(S):
            seen = (js <= pos + s).double()
            n = float(seen.sum())
            want = torch.zeros(D, dtype=torch.float64, device="cuda")
            want[:len(js)] = seen / max(n, 1)
            err = (o[s, 0].double() - want).abs().max()
            # (weights as fp16, the result as bf16)
            assert n == 0 or float(err) <= (2.0 ** -11 + 2.0 ** -8) / n, (i, s)
            if n:
                z = 40 + torch.tensor(n).double().log()
                assert bool((lse[s, 0].double() - z.cuda()).abs().max() <=
                            2.0 ** -15 * 41)


# ---- pages that the table names wrongly ----------------------------------------

def ref_without(a, hidden):
    """The attention with the keys hidden[b] left out, in 64 bits."""
    k, v = (torch.stack(dense(c, s, a["good"], a["group"]), 1)
            for c, s in ((a["kc"], a["ks"]), (a["vc"], a["vs"])))
    S, B, H, D = a["q"].shape
    T, _, Hk, _ = k.shape
    r = {n: torch.zeros((S, B, H, D)).double() for n in ("o", "A_o")}
    r["lse"] = torch.full((S, B, H), -float("inf")).double()
    r["X"] = torch.zeros((S, B, H)).double()
    for b in range(B):
        for s in range(S):
            for hk in range(Hk):
                js = [j for j in row_keys(a["ids"], b, s, hk,
                                          int(a["q_pos"][b]) + s, a["block"],
                                          a["local"], T) if j not in hidden[b]]
                if not js:
                    continue
                hs = slice(hk * (H // Hk), (hk + 1) * (H // Hk))
                qq = a["q"][s, b, hs].double()
                x = a["scale"] * qq @ k[js, b, hk].T
                p = torch.softmax(x, 1)
                r["o"][s, b, hs] = p @ v[js, b, hk]
                r["A_o"][s, b, hs] = p @ v[js, b, hk].abs()
                r["lse"][s, b, hs] = torch.logsumexp(x, 1)
                r["X"][s, b, hs] = (a["scale"] * qq.abs()
                                    @ k[js, b, hk].abs().T).amax(1)
    r["w_top"] = float(a["vs"].max())
    return r, T


@gpu
@pytest.mark.parametrize("case", [ATTN[1], ATTN[8], ATTN[9], ATTN[12],
                                  ATTN[15], ATTN[21]])
def test_rows_without_a_bad_page(dsa, case):
    """All rows of all sequences, with another wrong page in each."""
    a = attn_inputs(case, 24)
    B, pages, page = a["q"].shape[1], a["table"].shape[1], a["kc"].shape[1]
    a["good"] = a["table"].clone()
    hidden = []
    for b in range(B):
        bad = b % pages
        a["table"][b, bad] = (-1, a["kc"].shape[0], 2 ** 31 - 1)[b % 3]
        hidden.append(range(bad * page, (bad + 1) * page))
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) in (0, 6)
    r, T = ref_without(a, hidden)
    check_attn(r, o, lse, T)


# ---- other calls that the documentation allows ---------------------------------

@gpu
@pytest.mark.parametrize("shift", [0, 1])          # of the rows: 16-byte pieces
@pytest.mark.parametrize("S,D,R,group", [(1, 128, 128, 64), (3, 64, 32, 16),
                                         (90, 96, 64, 32)])
def test_append_far_away_with_a_rotation_scale(dsa, S, D, R, group, shift):
    """Positions near 2^30, scaled rotations, a batch that is broadcast; read
    back from there."""
    B, H, Hk, page = 2, 3, 2, 128
    far = 1 << 23                                  # pages of a sequence
    g = torch.Generator().manual_seed(5)
    n = (H + 2 * Hk) * D
    buf = torch.randn((S, 1, n + 8), generator=g).to(BF)
    cut = lambda t: t[..., shift:shift + n].unflatten(-1, (H + 2 * Hk, D)
                                                      ).expand(-1, B, -1, -1)
    q, k, v = cut(buf).split([H, Hk, Hk], 2)
    gq, gk, gv = cut(buf.cuda()).split([H, Hk, Hk], 2)
    kc, vc, ks, vs = make_cache(8, page, Hk, D, group, 8)
    start = torch.tensor([far * page - S - 3, far * page - 200])
    dev = [t.cuda() for t in (kc, vc, ks, vs)]
    table = torch.full((B, far), 99, dtype=torch.int32, device="cuda")
    table[:, -3:] = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32)
    wq, wk = weights(D, 3)
    m = 1.375
    st = start.to(torch.int32).cuda()
    out_q, ws = dsa.dsa_paged_append_q8(
        gk, gv, *dev, table, st, inv_freq=inv(R).cuda(), wk=wk.cuda(), eps=EPS,
        q=gq, wq=wq.cuda(), rot_scale=m)
    assert dsa.dsa_indexer_check(ws) == 0
    pos = start[None, :] + torch.arange(S)[:, None]
    want, mag = norm_rope_ref(k, wk, pos, inv(R), 0, False, EPS, m)
    base = (far - 3) * page                        # what the table's end names
    small, at = table[:, -3:].cpu(), (start - base).tolist()
    # 2^-19 of the pair for the norm and rotation, and the angle.  A turn's
    # fraction f / (2 pi) < 0.16 comes out of two roundings in 64 bits, 2^-53.5 of
    # it each at most: 2^30 positions later 2^-25 turns, 2^-22.3; the
    # definition's pos f is off by half a step at 2^30, 2^-24.  Both: below 2^-21.
    slack = 2.0 ** -19 * mag + 2.0 ** -21 * mag
    check_append(want, slack, kc, ks, dev[0].cpu(), dev[2].cpu(), small, at,
                 [S] * B, group)
    check_append(v.double(), 0.0, vc, vs, dev[1].cpu(), dev[3].cpu(), small, at,
                 [S] * B, group)
    want, mag = norm_rope_ref(q, wq, pos, inv(R), 0, False, EPS, m)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -19 + 2.0 ** -21) * mag + 1e-38
    assert bool(((out_q.double().cpu() - want).abs() <= tol).all())
    _, got, ws = dsa.dsa_paged_read_q8(*dev, table, S, first=st)
    assert dsa.dsa_indexer_check(ws) == 0
    full = dense(dev[1].cpu(), dev[3].cpu(), small, group)
    for b in range(B):
        assert torch.equal(got[:, b].double().cpu(), full[b][at[b]:at[b] + S])


@gpu
@pytest.mark.parametrize("case", [ATTN[1], ATTN[5], ATTN[8], ATTN[12],
                                  ATTN[15], ATTN[17]])
def test_attention_of_a_selection_alone(dsa, case):
    """No local blocks: a row's own block counts where it is named."""
    a = attn_inputs(case, 25)
    a["local"] = 0
    own = int(a["q_pos"][0]) // a["block"]
    a["ids"][0, ..., -1] = own
    o, lse, ws = call(dsa, a)
    assert dsa.dsa_indexer_check(ws) == 0
    r, T = reference(a)
    check_attn(r, o, lse, T)


@gpu
@pytest.mark.parametrize("topk", [0, 12])
@pytest.mark.parametrize("S,B,H,Hk,D,block", [(2100, 1, 6, 2, 64, 32),
                                              (1030, 2, 8, 1, 128, 128)])
def test_attention_of_long_chunks(dsa, S, B, H, Hk, D, block, topk):
    page, group, T = 256, 64, 4096
    a = long_cache(S, B, H, Hk, D, T, page, group, 26)
    g = torch.Generator(device="cuda").manual_seed(3)
    a["q_pos"] = torch.randint(0, T - S, (B,), generator=g, device="cuda"
                               ).to(torch.int32)
    ids = None
    if topk:
        ids = torch.randint(-1, T // block, (B, S, Hk, topk), generator=g,
                            device="cuda").to(torch.int32)
    o, lse = attend(dsa, a, ids, block)
    order = a["table"][0].long()
    k, v = ((a[c].double() * a[s].double().repeat_interleave(group, 1)[..., None]
             )[order].flatten(0, 1) for c, s in (("kc", "ks"), ("vc", "vs")))
    j = torch.arange(T, device="cuda")
    top = float(a["vs"].max())
    for b in range(B):
        pos = int(a["q_pos"][b]) + torch.arange(S, device="cuda")
        own = pos // block
        for h in range(H):
            hk = h // (H // Hk)
            sees = j[None] <= pos[:, None]
            if topk:
                held = torch.zeros((S, T // block + 1), dtype=torch.bool,
                                   device="cuda")
                i = ids[b, :, hk].long()
                held.scatter_(1, torch.where(i < 0, T // block, i), True)
                held[torch.arange(S), own] = True
                sees &= held[:, :-1].repeat_interleave(block, 1)
            x = 0.11 * a["q"][:, b, h].double() @ k[:, hk].T
            x = x.masked_fill(~sees, -float("inf"))
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            want, A = p @ v[:, hk], p @ v[:, hk].abs()
            tol = ((2.0 ** -11 + 2.0 ** -12) * A + 2.0 ** -8 * want.abs()
                   + T * 2.0 ** -22 * top + 1e-30)
            assert bool(((o[:, b, h].double() - want).abs() <= tol).all())
            X = (0.11 * a["q"][:, b, h].double().abs() @ k[:, hk].abs().T).amax(1)
            assert bool(((lse[:, b, h].double() - z).abs()
                         <= 2.0 ** -15 * (1 + X)).all())


@gpu
def test_more_than_2_to_the_31_steps(dsa):
    """Single tokens whose selections could have 2^31 steps of 32 keys between
    them: slices are counted in units of several.  Against the same blocks as
    short lists; a row's order of summation is another."""
    B, D, block, page, T = 33000, 64, 128, 4096, 1 << 21
    a = long_cache(1, 1, 1, 1, D, T, page, 128, 27)
    g = torch.Generator(device="cuda").manual_seed(4)
    a["q"] = torch.randn((1, B, 1, D), generator=g, device="cuda").to(BF)
    a["table"] = a["table"].repeat(B, 1)
    a["q_pos"] = torch.full((B,), T - 1, dtype=torch.int32, device="cuda")
    few = torch.randint(0, T // block - 1, (B, 1, 3), generator=g,
                        device="cuda").to(torch.int32)
    o, lse = attend(dsa, a, few, block)
    most = 16380
    assert B * (most + 1) * block // 32 > 2 ** 31
    ids = torch.full((B, 1, most), -1, dtype=torch.int32, device="cuda")
    ids[..., 7], ids[..., 9000], ids[..., -1] = few.unbind(-1)
    o2, lse2 = attend(dsa, a, ids, block)
    A, _ = attend(dsa, a, few, block, vc=(raw(a["vc"]) & 0x7f).view(E4M3))
    tol = (2 * (2.0 ** -11 + 2.0 ** -12) * A.double() * (1 + 2.0 ** -7)
           + 2 * 2.0 ** -8 * o.double().abs()
           + 2 * 4 * block * 2.0 ** -22 * float(a["vs"].max()))
    assert bool(((o2.double() - o.double()).abs() <= tol).all())
    assert bool(((lse2 - lse).abs() <= 2.0 ** -14 * (1 + lse.abs() + 40)).all())
