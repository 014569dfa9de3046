"""The 8-bit cache at the ends of its ranges: queries of any size, keys that
decide a long row, appends of every width, rows that are not finite.

Tolerances are those of tests/test_cache_q8.py (their sums are written down
there)."""
from __future__ import annotations

import pytest
import torch

from tests.cache_q8_ref import E4M3
from tests.test_cache_q8 import (ATTN, BF, attn_inputs, call, check_attn,
                                 dsa, raw, reference)  # noqa: F401

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
