"""Attention over selected blocks, contiguous and paged, forward and backward,
against the 64-bit definition (tests/block_ref.py holds the tolerances and
what they are made of), and the refusals of bad arguments."""
from __future__ import annotations

import math

import pytest
import torch

from tests.block_ref import (block_attn_ref, check_attn, check_grads,
                             row_keys)

gpu = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dsa():
    import dsa_sparse_attention_fwd_gb300 as m
    m.build()
    m.load_library()
    return m


def select(g, B, S, Hs, topk, nblk, empty=0.2):
    """Random ids with repeats and empty entries; some rows wholly empty."""
    ids = torch.randint(0, nblk, (B, S, Hs, topk), generator=g)
    ids[torch.rand(ids.shape, generator=g) < empty] = -1
    ids[torch.rand((B, S, Hs), generator=g) < 0.1] = -1
    return ids.to(torch.int32)


def problem(S, B, H, Hk, D, T, block, topk, shared, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((S, B, H, D), generator=g).to(BF)
    k = torch.randn((T, B, Hk, D), generator=g).to(BF)
    v = torch.randn((T, B, Hk, D), generator=g).to(BF)
    go = torch.randn((S, B, H, D), generator=g).to(BF)
    blocks = None
    if topk:
        blocks = select(g, B, S, 1 if shared else Hk, topk, -(-T // block))
        blocks = blocks[:, :, 0].contiguous() if shared else blocks
    return q, k, v, go, blocks


def cu(*ts):
    return [None if t is None else t.cuda() for t in ts]


CASES = [
    # S, B, H, Hk, D, T, block, topk, local, shared, q_pos
    (1, 1, 1, 1, 64, 1, 16, 1, 1, True, None),
    (1, 2, 4, 2, 128, 300, 64, 3, 1, False, [299, 17]),
    (130, 1, 16, 1, 128, 130, 64, 2, 1, True, None),
    (75, 2, 8, 4, 64, 75, 16, 3, 2, False, None),
    (70, 1, 10, 2, 64, 200, 32, 4, 0, False, [100]),       # rows without keys
    (33, 2, 12, 1, 128, 97, 16, 5, 1, True, [64, 0]),
    (40, 1, 64, 1, 128, 512, 128, 2, 1, True, [470]),      # 64 heads a group
    (67, 1, 3, 3, 128, 67, 32, 2, 1, False, None),         # one head a group
    (20, 1, 14, 2, 64, 333, 64, 0, 3, True, [313]),        # local blocks only
    (50, 2, 8, 2, 64, 40, 32, 2, 1, False, [-20, 30]),     # before and past the keys
    (260, 1, 4, 1, 64, 260, 16, 16, 1, True, None),
    (3, 1, 8, 1, 128, 4096, 16, 40, 2, True, [4093]),      # few rows, long list
]


@gpu
@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(dsa, case):
    S, B, H, Hk, D, T, block, topk, local, shared, q_pos = case
    q, k, v, go, blocks = problem(S, B, H, Hk, D, T, block, topk, shared, 11)
    scale = D ** -0.5
    qp = None if q_pos is None else torch.tensor(q_pos, dtype=torch.int32)
    dq, dk, dv, dgo, dbl, dqp = cu(q, k, v, go, blocks, qp)
    kw = dict(q_pos=dqp, local_blocks=local)
    o, lse, ws = dsa.dsa_block_attn_fwd(dq, dk, dv, dbl, block, scale, **kw)
    assert dsa.dsa_indexer_check(ws) == 0
    r = block_attn_ref(q, k, v, blocks, block, local, scale, qp, go)
    check_attn(r, o, lse)
    grads = dsa.dsa_block_attn_bwd(dq, dk, dv, o, lse, dgo, dbl, block, scale,
                                   **kw)
    assert dsa.dsa_indexer_check(grads[3]) == 0
    check_grads(r, *grads[:3])


@gpu
@pytest.mark.parametrize("case", [CASES[2], CASES[5], CASES[11]])
def test_same_bits_every_run(dsa, case):
    S, B, H, Hk, D, T, block, topk, local, shared, q_pos = case
    q, k, v, go, blocks = cu(*problem(S, B, H, Hk, D, T, block, topk, shared, 5))
    qp = None if q_pos is None else torch.tensor(q_pos, dtype=torch.int32).cuda()
    kw = dict(q_pos=qp, local_blocks=local)
    first = None
    for _ in range(3):
        o, lse, _ = dsa.dsa_block_attn_fwd(q, k, v, blocks, block, 0.1, **kw)
        g = dsa.dsa_block_attn_bwd(q, k, v, o, lse, go, blocks, block, 0.1, **kw)
        now = (o, lse) + g[:3]
        if first is None:
            first = now
        for a, b in zip(first, now):
            assert torch.equal(a, b)


@gpu
def test_backward_against_differences(dsa):
    """Directional differences of the 64-bit forward against the kernel's
    gradients: off by no more than the elements' tolerances add up to."""
    S, B, H, Hk, D, T, block, topk = 20, 1, 4, 2, 64, 40, 16, 2
    q, k, v, go, blocks = problem(S, B, H, Hk, D, T, block, topk, False, 3)
    qp = torch.tensor([20], dtype=torch.int32)
    dq, dk, dv, dgo, dbl, dqp = cu(q, k, v, go, blocks, qp)
    kw = dict(q_pos=dqp, local_blocks=1)
    o, lse, _ = dsa.dsa_block_attn_fwd(dq, dk, dv, dbl, block, 0.125, **kw)
    got = dsa.dsa_block_attn_bwd(dq, dk, dv, o, lse, dgo, dbl, block, 0.125,
                                 **kw)[:3]
    r = block_attn_ref(q, k, v, blocks, block, 1, 0.125, qp, go)
    g = torch.Generator().manual_seed(9)
    for _ in range(3):
        d = [torch.randn(t.shape, generator=g).double() for t in (q, k, v)]

        def loss(h):
            x = [t.double() + h * e for t, e in zip((q, k, v), d)]
            y = block_attn_ref(*x, blocks, block, 1, 0.125, qp)
            return float((y["o"] * go.double()).sum())
        h = 1e-4
        num = (loss(h) - loss(-h)) / (2 * h)
        ana = sum(float((a.double().cpu() * e).sum()) for a, e in zip(got, d))
        tol = sum(float(((r[t] * (1 + 2.0 ** -8) + 2.0 ** -8 * r[n].abs())
                         * e.abs()).sum())
                  for n, t, e in (("gq", "tq", d[0]), ("gk", "tk", d[1]),
                                  ("gv", "tv", d[2])))
        assert abs(num - ana) <= tol + 1e-6 * abs(num)


@gpu
def test_strided_and_broadcast_keys(dsa):
    """Keys and values read in place out of a fused projection's output, with
    heads outermost, and one sequence's shared by all."""
    S, B, H, Hk, D, T, block = 60, 3, 8, 2, 64, 60, 16
    q, k, v, go, blocks = problem(S, B, H, Hk, D, T, block, 2, False, 21)
    dq, dgo, dbl = cu(q, go, blocks)
    kw = dict(local_blocks=1)
    fused = torch.cat([k, v], dim=2).cuda()
    heads_first = k.permute(2, 1, 0, 3).contiguous().cuda().permute(2, 1, 0, 3)
    one_k, one_v = k[:, :1].expand_as(k), v[:, :1].expand_as(v)
    g1k = k[:, :1].contiguous().cuda().expand(-1, B, -1, -1)
    g1v = v[:, :1].contiguous().cuda().expand(-1, B, -1, -1)
    for name, rk, rv, gk, gv in (
            ("fused", k, v, fused[:, :, :Hk], fused[:, :, Hk:]),
            ("heads first", k, v, heads_first, v.cuda()),
            ("broadcast", one_k, one_v, g1k, g1v)):
        o, lse, _ = dsa.dsa_block_attn_fwd(dq, gk, gv, dbl, block, 0.125, **kw)
        r = block_attn_ref(q, rk, rv, blocks, block, 1, 0.125, None, go)
        check_attn(r, o, lse)
        grads = dsa.dsa_block_attn_bwd(dq, gk, gv, o, lse, dgo, dbl, block,
                                       0.125, **kw)
        check_grads(r, *grads[:3])


PAGED = [
    # S, B, H, Hk, D, block, page, max_pages, topk, local, shared, q_pos
    (1, 3, 8, 2, 128, 64, 64, 9, 4, 1, False, [0, 300, 575]),
    (1, 2, 5, 1, 64, 16, 64, 40, 60, 2, True, [2559, 700]),
    (4, 2, 16, 4, 64, 32, 128, 6, 3, 1, False, [200, 764]),
    (70, 1, 20, 2, 128, 128, 256, 4, 2, 2, True, [900]),
    (2, 1, 64, 1, 128, 16, 16, 30, 8, 0, True, [470]),
    (1, 40, 32, 4, 128, 64, 64, 33, 16, 1, False, list(range(40, 2040, 50))),
]


@gpu
@pytest.mark.parametrize("case", PAGED)
@pytest.mark.parametrize("heads_first", [False, True])
def test_paged(dsa, case, heads_first):
    S, B, H, Hk, D, block, page, mp, topk, local, shared, q_pos = case
    T = page * mp
    q, k, v, _, blocks = problem(S, B, H, Hk, D, T, block, topk, shared, 31)
    qp = torch.tensor(q_pos, dtype=torch.int32)
    r = block_attn_ref(q, k, v, blocks, block, local, D ** -0.5, qp)
    # the cache: pages in random order among others that hold NaN, as do the
    # slots past each sequence's last row, and the pages that no row needs
    # have no id
    g = torch.Generator().manual_seed(1)
    P = B * mp + 2
    perm = torch.randperm(P, generator=g)[:B * mp].view(B, mp)
    kc = torch.full((P, page, Hk, D), math.nan, dtype=BF)
    vc = torch.full((P, page, Hk, D), math.nan, dtype=BF)
    for b in range(B):
        n = int(qp[b]) + S
        kk, vv = k[:, b].clone(), v[:, b].clone()
        kk[n:], vv[n:] = math.nan, math.inf
        kc[perm[b]] = kk.view(mp, page, Hk, D)
        vc[perm[b]] = vv.view(mp, page, Hk, D)
        perm[b, -(-n // page):] = -1
    if heads_first:
        kc, vc = kc.transpose(1, 2).contiguous(), vc.transpose(1, 2).contiguous()
    dq, dkc, dvc, dt, dbl, dqp = cu(q, kc, vc, perm.to(torch.int32), blocks, qp)
    if heads_first:
        dkc, dvc = dkc.transpose(1, 2), dvc.transpose(1, 2)
    o, lse, ws = dsa.dsa_block_attn_paged_fwd(
        dq, dkc, dvc, dt, dbl, block, D ** -0.5, q_pos=dqp,
        local_blocks=local)
    assert dsa.dsa_indexer_check(ws) == 0
    check_attn(r, o, lse)


@gpu
@pytest.mark.parametrize("what", ["nan", "inf", "lowest"])
def test_masked_values_do_not_reach_a_row(dsa, what):
    """Special values in a block that only some rows of a tile attend to, and
    in keys that only later rows see, change those rows alone."""
    S, B, H, Hk, D, T, block = 48, 1, 4, 1, 64, 96, 16
    q, k, v, _, _ = problem(S, B, H, Hk, D, T, block, 0, True, 41)
    qp = torch.tensor([48], dtype=torch.int32)
    blocks = torch.zeros((B, S, 2), dtype=torch.int32)
    blocks[:, :, 1] = 1
    blocks[:, ::3, 1] = 2                  # every third row holds block 2
    bad = {"nan": math.nan, "inf": math.inf,
           "lowest": torch.finfo(BF).min}[what]
    k2, v2 = k.clone(), v.clone()
    v2[40] = bad
    k2[41] = bad
    v2[48 + 37] = bad                      # the row 37's own key
    r = block_attn_ref(q, k, v, blocks, block, 1, 0.125, qp)
    run = lambda kk, vv: dsa.dsa_block_attn_fwd(
        *cu(q, kk, vv, blocks), block, 0.125, q_pos=qp.cuda(), local_blocks=1)
    o, lse, _ = run(k2, v2)
    clean = torch.ones(S, dtype=torch.bool)
    clean[::3] = False
    clean[37:] = False
    pick = lambda t: t[clean]
    check_attn({n: pick(t) for n, t in r.items()}, pick(o.cpu()), pick(lse.cpu()))
    if what != "lowest":
        assert not bool(torch.isfinite(o[0::3].float()).all(-1).any())
        assert not bool(torch.isfinite(o[37].float()).all(-1).any())


@gpu
def test_large_scores(dsa):
    """Scores far beyond exp's range: the running maximum carries them."""
    q, k, v, go, blocks = problem(64, 1, 8, 2, 64, 64, 16, 3, False, 51)
    q = (q.float() * 60).to(BF)
    o, lse, _ = dsa.dsa_block_attn_fwd(*cu(q, k, v, blocks), 16, 0.5,
                                       local_blocks=1)
    r = block_attn_ref(q, k, v, blocks, 16, 1, 0.5, None)
    lse64 = r["lse"][r["lse"] > -math.inf]
    assert float(lse64.max()) > 500
    # a score of 1000 carries 2^-24 of itself per accumulation step: its
    # exponential's relative error is the score's absolute one
    err = 2.0 ** -20 * r["X"][..., None]
    tol = ((2.0 ** -8 + 2.0 ** -12) + 2 * err) * r["A_o"] + 2.0 ** -8 * r["o"].abs()
    assert bool(((o.double().cpu() - r["o"]).abs() <= tol + 1e-30).all())
    d = (lse.double().cpu() - r["lse"]).abs()
    d = torch.where(r["lse"] == -math.inf, torch.zeros_like(d), d)
    assert bool((d <= 2.0 ** -15 * (1 + r["X"])).all())


@gpu
def test_reports_bad_ids_and_pages(dsa):
    q, k, v, _, blocks = problem(8, 1, 4, 1, 64, 64, 16, 2, True, 61)
    bad = blocks.clone()
    bad[0, 3, 0] = 4                       # one past the last block
    good = blocks.clone()
    good[0, 3, 0] = -1
    qp = torch.tensor([50], dtype=torch.int32)
    run = lambda bl: dsa.dsa_block_attn_fwd(*cu(q, k, v, bl), 16, 0.125,
                                            q_pos=qp.cuda(), local_blocks=1)
    o1, l1, w1 = run(bad)
    o2, l2, w2 = run(good)
    assert dsa.dsa_indexer_check(w1) == 6
    assert dsa.dsa_indexer_check(w1) == 0
    assert dsa.dsa_indexer_check(w2) == 0
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    # a page id outside the cache: its blocks are skipped
    kc, vc = k.view(4, 16, 1, 64), v.view(4, 16, 1, 64)
    for wrong in (-1, 4, 2 ** 31 - 1):
        table = torch.tensor([[0, 1, wrong, 3]], dtype=torch.int32)
        blocks = torch.tensor([[[0, 2]]], dtype=torch.int32)
        less = torch.tensor([[[0, -1]]], dtype=torch.int32)
        qp1 = torch.tensor([63], dtype=torch.int32)
        o, lse, ws = dsa.dsa_block_attn_paged_fwd(
            *cu(q[:1], kc, vc, table, blocks), 16, 0.125, q_pos=qp1.cuda(),
            local_blocks=1)
        assert dsa.dsa_indexer_check(ws) == 6
        r = block_attn_ref(q[:1], k, v, less, 16, 1, 0.125, qp1)
        check_attn(r, o, lse)


@gpu
def test_paged_past_32_bit_offsets(dsa):
    """Pages beyond 2^31 elements."""
    page, Hk, D = 64, 8, 128
    pages = 2 ** 31 // (page * Hk * D) + 3
    kc = torch.zeros((pages, page, Hk, D), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    q, k, v, _, _ = problem(1, 1, 16, Hk, D, 2 * page, 64, 0, True, 71)
    ids = [pages - 1, pages - 3]
    kc[ids] = k.cuda().view(2, page, Hk, D)
    vc[ids] = v.cuda().view(2, page, Hk, D)
    table = torch.tensor([ids], dtype=torch.int32)
    blocks = torch.tensor([[[0]]], dtype=torch.int32)
    qp = torch.tensor([100], dtype=torch.int32)
    o, lse, ws = dsa.dsa_block_attn_paged_fwd(
        q.cuda(), kc, vc, table.cuda(), blocks.cuda(), 64, 0.1,
        q_pos=qp.cuda(), local_blocks=1)
    assert dsa.dsa_indexer_check(ws) == 0
    check_attn(block_attn_ref(q, k, v, blocks, 64, 1, 0.1, qp), o, lse)


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_the_longest_context(dsa, D):
    """16384 blocks: the block words take most of the shared memory, and the
    ids that are 16 bits wide on the way reach their end."""
    S, H, Hk, block, T = 5, 12, 1, 16, 16384 * 16
    g = torch.Generator().manual_seed(101)
    q = torch.randn((S, 1, H, D), generator=g).to(BF)
    go = torch.randn((S, 1, H, D), generator=g).to(BF)
    k = torch.randn((T, 1, Hk, D), generator=g).to(BF)
    v = torch.randn((T, 1, Hk, D), generator=g).to(BF)
    blocks = torch.randint(0, 16384, (1, S, 9), generator=g, dtype=torch.int32)
    blocks[0, :, 0] = 16383
    blocks[0, :, 1] = 0
    qp = torch.tensor([T - 3], dtype=torch.int32)     # rows past the last key
    dq, dk, dv, dgo, dbl, dqp = cu(q, k, v, go, blocks, qp)
    kw = dict(q_pos=dqp, local_blocks=2)
    o, lse, ws = dsa.dsa_block_attn_fwd(dq, dk, dv, dbl, block, 0.125, **kw)
    assert dsa.dsa_indexer_check(ws) == 0
    r = block_attn_ref(q, k, v, blocks, block, 2, 0.125, qp, go)
    check_attn(r, o, lse)
    grads = dsa.dsa_block_attn_bwd(dq, dk, dv, o, lse, dgo, dbl, block, 0.125,
                                   **kw)
    assert dsa.dsa_indexer_check(grads[3]) == 0
    check_grads(r, *grads[:3])


@gpu
def test_one_workspace_for_many_calls(dsa):
    """A workspace that is zeroed once serves calls of other shapes, split and
    not, forward and backward, and a call that reports an error."""
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    for rnd in range(2):
        for case in (CASES[11], CASES[1], CASES[2], CASES[8]):
            S, B, H, Hk, D, T, block, topk, local, shared, q_pos = case
            q, k, v, go, blocks = cu(*problem(S, B, H, Hk, D, T, block, topk,
                                              shared, 111))
            qp = None
            if q_pos is not None:
                qp = torch.tensor(q_pos, dtype=torch.int32).cuda()
            kw = dict(q_pos=qp, local_blocks=local)
            o, lse, _ = dsa.dsa_block_attn_fwd(q, k, v, blocks, block, 0.1, **kw)
            o2, lse2, _ = dsa.dsa_block_attn_fwd(q, k, v, blocks, block, 0.1,
                                                 workspace=ws, **kw)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
            g = dsa.dsa_block_attn_bwd(q, k, v, o, lse, go, blocks, block, 0.1,
                                       **kw)
            g2 = dsa.dsa_block_attn_bwd(q, k, v, o, lse, go, blocks, block,
                                        0.1, workspace=ws, **kw)
            assert all(torch.equal(a, b) for a, b in zip(g[:3], g2[:3]))
            assert dsa.dsa_indexer_check(ws) == 0
        # other entry points write the rest of it
        x = torch.ones((64, 2, 4, 128), device="cuda")
        w1 = torch.ones(128, device="cuda")
        dsa.dsa_norm_rope_bwd(x, None, x, None, None, wq=w1, workspace=ws)
        qi = torch.ones((40, 1, 4, 64), dtype=BF, device="cuda")
        dsa.dsa_indexer_fwd(qi, qi[:, :, 0].contiguous(),
                            torch.ones((40, 1, 4), device="cuda"), 1, 8,
                            workspace=ws)
        q, k, v, _, blocks = problem(1, 1, 4, 1, 64, 2048, 16, 16, True, 5)
        blocks[0, 0, 3] = 5000
        dsa.dsa_block_attn_fwd(*cu(q, k, v, blocks), 16, 0.1, workspace=ws,
                               q_pos=torch.tensor([2047]).int().cuda())
        assert dsa.dsa_indexer_check(ws) == 6


@gpu
@pytest.mark.parametrize("D,G,block", [(64, 1, 16), (128, 4, 64)])
@pytest.mark.parametrize("first", [None, -2])
def test_gradients_of_rows_with_few_keys(dsa, D, G, block, first):
    """At a sequence's first positions the weights are one-sided and dS is a
    small difference: the rounding of o does not enter it.  Errors: dS's
    rounding, 2^-8 of it; a score of magnitude X is a chain of up to nine fp32
    sums, 9 2^-23 X off, and so is the log-sum: P is 2^-18 (1 + X) off with
    the exponential's 2^-21, and so is what dS is made of; then the result's
    rounding."""
    S, B, Hk = 40, 2, 2
    q, k, v, go, blocks = problem(S, B, Hk * G, Hk, D, S, block, 3, False, 17)
    qp = None if first is None else torch.tensor([first, 0], dtype=torch.int32)
    kw = dict(q_pos=None if qp is None else qp.cuda(), local_blocks=1)
    dq, dk, dv, dgo, dbl = cu(q, k, v, go, blocks)
    o, lse, _ = dsa.dsa_block_attn_fwd(dq, dk, dv, dbl, block, 0.2, **kw)
    gq = dsa.dsa_block_attn_bwd(dq, dk, dv, o, lse, dgo, dbl, block, 0.2,
                                **kw)[0].double().cpu()
    r = block_attn_ref(q, k, v, blocks, block, 1, 0.2, qp, go)
    for b in range(B):
        p0 = 0 if qp is None else int(qp[b])
        for s in range(max(0, -p0), 32 - p0):
            for h in range(Hk * G):
                hk = h // G
                js = row_keys(blocks, b, s, hk, p0 + s, block, 1, S)
                kk, vv = k[js, b, hk].double(), v[js, b, hk].double()
                g = go[s, b, h].double()
                p = torch.softmax(0.2 * kk @ q[s, b, h].double(), 0)
                dp = vv @ g
                ds = 0.2 * p * (dp - p @ dp)
                mag = vv.abs() @ g.abs()
                off = 2.0 ** -18 * (1 + float(r["X"][s, b, h]))
                e = 2.0 ** -8 * ds.abs() + 0.2 * p * off * (mag + p @ mag)
                tol = e @ kk.abs()
                want = r["gq"][s, b, h]
                tol = tol + 2.0 ** -8 * (want.abs() + tol) + 1e-30
                err = (gq[s, b, h] - want).abs()
                assert bool((err <= tol).all()), (b, s, h, (err / tol).max())


@gpu
def test_agrees_with_the_indexers_selection(dsa):
    """The indexer's top-k over keys compressed by the block size names the
    blocks: together they are attention over the best whole blocks and the
    row's own."""
    S, H, Hk, D, block, topk = 128, 8, 2, 64, 16, 3
    q, k, v, _, _ = problem(S, 1, H, Hk, D, S, block, 0, True, 81)
    g = torch.Generator().manual_seed(82)
    qi = torch.randn((S, 1, 4, 32), generator=g).to(BF)
    ki = torch.randn((S // block, 1, 32), generator=g).to(BF)
    w = torch.rand((S, 1, 4), generator=g)
    _, idx = dsa.v4_lighting_indexer(*cu(qi, ki, w), block, topk)
    o, lse, _ = dsa.dsa_block_attn_fwd(*cu(q, k, v), idx, block, 0.125,
                                       local_blocks=1)
    r = block_attn_ref(q, k, v, idx.cpu(), block, 1, 0.125)
    check_attn(r, o, lse)


@gpu
def test_other_stream_and_graph(dsa):
    q, k, v, go, blocks = cu(*problem(64, 1, 16, 2, 64, 64, 16, 2, False, 91))
    kw = dict(local_blocks=1)
    o, lse, ws = dsa.dsa_block_attn_fwd(q, k, v, blocks, 16, 0.125, **kw)
    g = dsa.dsa_block_attn_bwd(q, k, v, o, lse, go, blocks, 16, 0.125, **kw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        o2, lse2, _ = dsa.dsa_block_attn_fwd(q, k, v, blocks, 16, 0.125, **kw)
        g2 = dsa.dsa_block_attn_bwd(q, k, v, o2, lse2, go, blocks, 16, 0.125,
                                    **kw)
    st.synchronize()
    outs = [torch.zeros_like(t) for t in (o, lse, *g[:3])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_block_attn_fwd(q, k, v, blocks, 16, 0.125, out_o=outs[0],
                               out_lse=outs[1], workspace=ws, **kw)
        dsa.dsa_block_attn_bwd(q, k, v, outs[0], outs[1], go, blocks, 16,
                               0.125, grad_q=outs[2], grad_k=outs[3],
                               grad_v=outs[4], workspace=g[3], **kw)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip((o, lse, *g[:3]), (o2, lse2, *g2[:3]), outs):
        assert torch.equal(a, b) and torch.equal(a, c)


# ---- refusals (no GPU) --------------------------------------------------------

def test_calls_refuse_host_tensors(dsa):
    q, k, v, go, blocks = problem(4, 1, 2, 1, 64, 16, 16, 1, True, 1)
    lse = torch.zeros((4, 1, 2))
    with pytest.raises(ValueError, match="CUDA tensor"):
        dsa.dsa_block_attn_fwd(q, k, v, blocks, 16, 0.1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dsa.dsa_block_attn_bwd(q, k, v, q, lse, go, blocks, 16, 0.1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dsa.dsa_block_attn_paged_fwd(
            q, k.view(1, 16, 1, 64), v.view(1, 16, 1, 64),
            torch.zeros((1, 1), dtype=torch.int32), blocks, 16, 0.1)


FAKE = 1 << 20  # aligned, never read: every case fails before its use
REFUSALS = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(blocks=None), 1), (dict(o=None), 1), (dict(lse=None), 1),
    (dict(S=0), 1), (dict(H=3), 1), (dict(Hk=0), 1), (dict(topk=-1), 1),
    (dict(topk=0, local=0), 1), (dict(sel=3), 1), (dict(scale=0.0), 1),
    (dict(scale=math.nan), 1), (dict(D=96), 2), (dict(blk=48), 2),
    (dict(blk=256), 2), (dict(H=130), 2), (dict(ws=None), 3),
    (dict(wsb=16), 3), (dict(ws=FAKE + 64), 1), (dict(q=FAKE + 8), 1),
    (dict(k=FAKE + 2), 1), (dict(o=FAKE + 8), 1), (dict(blocks=FAKE + 2), 1),
]


@pytest.mark.parametrize("over,code", REFUSALS + [
    (dict(T=0), 1), (dict(T=16 * 16384 + 1, blk=16), 2),
    (dict(strides=(60, 64, 64, 128, 64, 64)), 1),
    (dict(strides=(128, 64, 64, 128, -64, 64)), 1),
])
def test_forward_refuses(dsa, over, code):
    import ctypes
    a = dict(q=FAKE, k=FAKE, v=FAKE, strides=None, S=4, B=1, H=4, Hk=2, D=64,
             T=64, blocks=FAKE, sel=1, topk=2, blk=16, local=1, qp=None,
             scale=0.1, o=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40, st=None)
    a.update(over)
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_int64 * 6)(*a["strides"])
    assert dsa.load_library().dsa_block_attn_fwd(*a.values()) == code


@pytest.mark.parametrize("over,code", REFUSALS + [
    (dict(table=None), 1), (dict(pages=0), 1), (dict(page=0), 1),
    (dict(maxp=0), 1), (dict(page=24), 2), (dict(maxp=1 << 30), 2),
    (dict(table=FAKE + 1), 1),
])
def test_paged_refuses(dsa, over, code):
    a = dict(q=FAKE, k=FAKE, v=FAKE, strides=None, pages=9, page=256,
             table=FAKE, maxp=4, S=4, B=1, H=4, Hk=2, D=64, blocks=FAKE, sel=1,
             topk=2, blk=16, local=1, qp=None, scale=0.1, o=FAKE, lse=FAKE,
             ws=FAKE, wsb=1 << 40, st=None)
    a.update(over)
    if over.get("blk") == 256:
        a["page"] = 256
    assert dsa.load_library().dsa_block_attn_paged_fwd(*a.values()) == code


@pytest.mark.parametrize("over,code", REFUSALS + [
    (dict(go=None), 1), (dict(gq=None), 1), (dict(gk=None), 1),
    (dict(gv=None), 1), (dict(gk=FAKE + 4), 1), (dict(go=FAKE + 2), 1),
])
def test_backward_refuses(dsa, over, code):
    a = dict(q=FAKE, k=FAKE, v=FAKE, strides=None, o=FAKE, lse=FAKE, go=FAKE,
             S=4, B=1, H=4, Hk=2, D=64, T=64, blocks=FAKE, sel=1, topk=2,
             blk=16, local=1, qp=None, scale=0.1, gq=FAKE, gk=FAKE, gv=FAKE,
             ws=FAKE, wsb=1 << 40, st=None)
    a.update(over)
    assert dsa.load_library().dsa_block_attn_bwd(*a.values()) == code


@pytest.mark.parametrize("args", [
    (0, 1, 4, 2, 64, 64, 16, 1, 1), (4, 1, 3, 2, 64, 64, 16, 1, 1),
    (4, 1, 4, 0, 64, 64, 16, 1, 1), (4, 1, 4, 2, 64, 0, 16, 1, 1),
    (4, 1, 4, 2, 64, 64, 0, 1, 1),
])
def test_workspace_size_of_invalid_shapes(dsa, args):
    assert dsa.dsa_block_attn_workspace_size(*args) == 0
    assert dsa.dsa_block_attn_bwd_workspace_size(*args) == 0


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,G", [(1, 4), (1, 1), (20, 16)])
@pytest.mark.parametrize("n", [1, 3, 5])
def test_ragged_blocks_whatever_shared_memory_holds(dsa, D, S, G, n):
    """Blocks of 16 in a step of 64: the rows of keys that the last step does
    not load are numbers, so NaN that an earlier kernel left in shared memory
    changes no bit.  No key comes after a row's position here: those would be
    hidden one by one."""
    B, Hk, T, block = 300, 1, 160, 16
    q, k, v, _, _ = problem(S, B, Hk * G, Hk, D, T, block, 0, True, 121)
    blocks = torch.arange(n, dtype=torch.int32).expand(B, S, n).contiguous()
    qp = torch.full((B,), 100, dtype=torch.int32)
    dq, dk, dv, dbl, dqp = cu(q, k, v, blocks, qp)
    # at least 304 tiles of three blocks: every SM's shared memory, and keys in
    # the stages where this call's go
    if G * S <= 32:
        shape, rows, first = (1, 640, 32, D), 192, 191
    else:
        shape, rows, first = (640, 1, 64, D), 640, 0
    fq = torch.ones(shape, dtype=BF, device="cuda")
    fp = torch.full((shape[1],), first, dtype=torch.int32, device="cuda")
    fill = {name: torch.full((rows, shape[1], 1, D), x, dtype=BF, device="cuda")
            for name, x in (("zero", 0.0), ("nan", math.nan))}
    run = lambda: dsa.dsa_block_attn_fwd(dq, dk, dv, dbl, block, 0.125,
                                         q_pos=dqp)[:2]
    got = {}
    for name, x in fill.items():
        dsa.dsa_block_attn_fwd(fq, x, x, None, 64, 0.1, q_pos=fp,
                               local_blocks=3)
        got[name] = run()
    assert torch.equal(got["zero"][0], got["nan"][0])
    assert torch.equal(got["zero"][1], got["nan"][1])
    sub = slice(0, 2)
    r = block_attn_ref(q[:, sub], k[:, sub], v[:, sub], blocks[sub], block, 0,
                       0.125, qp)
    check_attn(r, got["nan"][0][:, sub], got["nan"][1][:, sub])


@gpu
@pytest.mark.parametrize("D,G,block", [(64, 1, 16), (64, 4, 64), (128, 4, 16),
                                       (128, 12, 32)])
def test_gradients_of_one_sided_rows(dsa, D, G, block):
    """A sink key that every row holds, with most of the weight of many: dS is
    a small difference there, and the rounding of o in delta does not enter it
    as a whole.  With d the key of more than half of the weight (if any) and
    delta0 = do.o from the rounded o, off by e0 <= 2^-8 sum |do o|:
      dS_j: its rounding, 2^-8 of it; P is off by a factor 1 + 2^-18 (1 + X)
    (the exponential, and a score's and the log-sum's chains of nine fp32
    sums), which also reaches delta = sum P (dP - delta0) + delta0; dP and
    delta0 by 2^-20 of their magnitudes;
      dq, where d exists: dS_d is minus the others' sum, so e0 reaches the
    others only, P_j e0 (|k_j| + |k_d|); else P_j e0 |k_j|;
      the results' rounding."""
    S, B, Hk, T, first = 96, 1, 2, 140, 44
    q, k, v, go, blocks = problem(S, B, Hk * G, Hk, D, T, block, 3, False, 131)
    g = torch.Generator().manual_seed(132)
    u = torch.randn(D, generator=g)
    u *= 9 ** 0.5 * D ** 0.25 / u.norm()
    q = (q.float() + u).to(BF)
    k[3] = (k[3].float() + u).to(BF)
    blocks[..., 0] = 0
    qp = torch.tensor([first], dtype=torch.int32)
    scale = D ** -0.5
    kw = dict(q_pos=qp.cuda(), local_blocks=1)
    dq, dk, dv, dgo, dbl = cu(q, k, v, go, blocks)
    o, lse, _ = dsa.dsa_block_attn_fwd(dq, dk, dv, dbl, block, scale, **kw)
    grads = dsa.dsa_block_attn_bwd(dq, dk, dv, o, lse, dgo, dbl, block, scale,
                                   **kw)[:3]
    r = block_attn_ref(q, k, v, blocks, block, 1, scale, qp, go)
    tq, tk = torch.zeros_like(r["tq"]), torch.zeros_like(r["tk"])
    sided = 0
    for s in range(S):
        for h in range(Hk * G):
            hk = h // G
            js = row_keys(blocks, 0, s, hk, first + s, block, 1, T)
            kk, vv = k[js, 0, hk].double(), v[js, 0, hk].double()
            qq, gg = q[s, 0, h].double(), go[s, 0, h].double()
            p = torch.softmax(scale * kk @ qq, 0)
            dp = vv @ gg
            gap = (dp - p @ dp).abs()
            e0 = 2.0 ** -8 * float(gg.abs() @ (p @ vv).abs())
            mag = vv.abs() @ gg.abs()
            off = 2.0 ** -18 * (1 + float(r["X"][s, 0, h]))
            e = scale * p * ((2.0 ** -8 + off) * gap + off * (p @ gap + e0)
                             + 2.0 ** -20 * (mag + p @ mag))
            tk[js, 0, hk] += e[:, None] * qq.abs()
            top = int(p.argmax())
            few = e + scale * p * e0                # e0 in every key
            t = few @ kk.abs()
            if p[top] > 0.5 - 2.0 ** -10:
                few[top] = 2.0 ** -18 * scale * e0  # what cancels, in fp32
                both = few @ (kk.abs() + kk[top].abs())
                t = both if p[top] > 0.5 + 2.0 ** -10 else torch.maximum(t, both)
            tq[s, 0, h] = t
            sided += int(p[top] > 0.95)
    assert sided > 0.2 * S * Hk * G
    check_grads(dict(r, tq=tq, tk=tk), *grads)


def test_backward_limits(dsa):
    """The backward's own limits are those of the selection at hand, and
    reported as what they are."""
    lib = dsa.load_library()
    a = dict(q=FAKE, k=FAKE, v=FAKE, strides=None, o=FAKE, lse=FAKE, go=FAKE,
             S=4, B=64, H=8, Hk=8, D=64, T=1 << 18, blocks=FAKE, sel=1, topk=2,
             blk=64, local=1, qp=None, scale=0.1, gq=FAKE, gk=FAKE, gv=FAKE,
             ws=FAKE, wsb=16, st=None)
    call = lambda **over: lib.dsa_block_attn_bwd(*dict(a, **over).values())
    # 2^17 lists of key tiles where the heads share a selection, 2^20 where not:
    # (a small workspace, so that what is supported is refused for that)
    assert call() == 3
    assert call(sel=8) == 2
    size = dsa.dsa_block_attn_bwd_workspace_size
    assert size(4, 64, 8, 8, 64, 1 << 18, 64, 2, 1) > 0
    assert size(4, 1024, 8, 8, 64, 1 << 18, 64, 2, 1) == 0
    assert call(B=1024) == 2
    # launches of more than 2^31 CTAs
    assert call(S=1, B=1 << 19, H=1024, Hk=64, T=128, topk=1) == 2
    assert call(S=1, B=1 << 17, H=1024, Hk=1024, T=128, topk=1) == 2


def test_backward_reports_unsupported_shapes(dsa, monkeypatch):
    """A valid shape past the limits is unsupported, not invalid; refused
    before its (host) tensors are read."""
    monkeypatch.setattr(dsa, "_on_gpu", lambda *a: 0)
    monkeypatch.setattr(dsa, "_raw_stream", lambda *a: None)
    S, B, Hk, D = 1, 1 << 17, 8, 64
    x = torch.empty((S, B, Hk, D), dtype=BF)
    lse = torch.empty((S, B, Hk))
    blocks = torch.empty((B, S, Hk, 1), dtype=torch.int32)
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_block_attn_bwd(x, x, x, x, lse, x, blocks, 16, 0.1)
    assert e.value.code == 2
