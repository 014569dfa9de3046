"""Per-head norm with rotation, its backward, and the append to a paged cache
against 64-bit definitions, and the refusals of bad arguments.

Tolerances: half a step of the output's type (finfo.eps / 2) of the value,
plus 2^-19 of the rotated pair's magnitude for fp32: the mean of squares and
its root (below 2^-21), four products (2^-22), the angle (rounded to 2^-25
turns, 2^-22 rad) and sine and cosine (2^-23).  Backward: twice the chain of
products and two sums, 2^-17 of the magnitudes; the weights' gradient sums at
most 600 terms in one accumulator: 2^-14.
"""
from __future__ import annotations

import math

import pytest
import torch

from tests.block_ref import (norm_rope_bwd_ref, norm_rope_ref, rotate_ref)

gpu = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def dsa():
    import dsa_sparse_attention_fwd_gb300 as m
    m.build()
    m.load_library()
    return m


def make(S, B, H, D, dt, seed, fused):
    g = torch.Generator().manual_seed(seed)
    if fused:  # rows inside a wider buffer
        buf = torch.randn((S, B, H * D + 24), generator=g).to(dt)
        return buf[..., 8:8 + H * D].unflatten(-1, (H, D))
    return torch.randn((S, B, H, D), generator=g).to(dt)


def on_gpu(x):
    """The tensor on the GPU with its strides kept."""
    if x is None:
        return None
    if x._base is None or x.is_contiguous():
        return x.cuda()
    return x._base.cuda().as_strided(x.shape, x.stride(), x.storage_offset())


CASES = [
    # S, B, H, Hk, D, R, r0, interleaved, dtype, fused
    (1, 1, 1, 1, 8, 8, 0, True, torch.bfloat16, False),
    (5, 3, 4, 2, 128, 128, 0, False, torch.bfloat16, False),
    (7, 2, 5, 1, 128, 64, 64, True, torch.bfloat16, True),
    (33, 1, 8, 8, 64, 32, 0, False, torch.float16, True),
    (3, 2, 3, 1, 256, 256, 0, False, torch.float32, False),
    (4, 2, 6, 2, 192, 64, 128, False, torch.float32, True),
    (6, 1, 7, 3, 96, 96, 0, True, torch.float16, False),
    # odd sizes: no 16-byte pieces
    (5, 2, 3, 1, 50, 12, 3, False, torch.bfloat16, False),
    (5, 1, 2, 2, 66, 66, 0, True, torch.float32, False),
    (2, 2, 1, 1, 2, 2, 0, False, torch.bfloat16, False),
    (4, 1, 2, 1, 250, 20, 230, True, torch.float16, False),
    # halves that do not fall on 16-byte pieces
    (4, 1, 2, 1, 64, 24, 8, False, torch.bfloat16, False),
    # many tokens
    (700, 2, 4, 2, 64, 64, 0, False, torch.bfloat16, True),
]


def inv(R):
    i = torch.arange(R // 2, dtype=torch.float64)
    return 10000.0 ** (-2 * i / R)


def positions(S, B, seed):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(-5, 4000, (S, B), generator=g, dtype=torch.int32)
    pos.view(-1)[0] = 2 ** 31 - 1           # as exact as any other
    pos.view(-1)[-1] = 1048577
    return pos


def weights(D, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(D, generator=g),
            1 + 0.3 * torch.randn(D, generator=g))


def assert_close(name, got, want, mag, dt, rel):
    got = got.double().cpu()
    tol = torch.finfo(dt).eps / 2 * want.abs() + rel * mag + (
        2.0 ** -25 if dt == torch.float16 else 1e-38)   # smallest fp16 step
    err = (got - want).abs()
    assert bool((err <= tol).all()), f"{name}: {(err / tol).max():.3g} tol"


# The reference's own angle: pos * inv_freq in 64 bits is off by 2^-53 of
# the angle, 2^-22 rad at 2^31: inside the bound.
@gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("normed", ["both", "q", "none"])
def test_forward(dsa, case, normed):
    S, B, H, Hk, D, R, r0, inter, dt, fused = case
    q, k = make(S, B, H, D, dt, 1, fused), make(S, B, Hk, D, dt, 2, fused)
    wq, wk = weights(D, 3)
    wq = None if normed == "none" else wq
    wk = wk if normed == "both" else None
    pos, f = positions(S, B, 4), inv(R)
    oq, ok = dsa.dsa_norm_rope_fwd(
        on_gpu(q), on_gpu(k), f.cuda(), positions=pos.cuda(),
        wq=on_gpu(wq), wk=on_gpu(wk), eps=EPS, rot_start=r0,
        interleaved=inter, rot_scale=1.25)
    for name, x, w, got in (("q", q, wq, oq), ("k", k, wk, ok)):
        want, mag = norm_rope_ref(x, w, pos, f, r0, inter, EPS, 1.25)
        assert_close(name, got, want, mag, dt, 2.0 ** -19)


@gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("normed", ["both", "k", "none"])
def test_backward(dsa, case, normed):
    S, B, H, Hk, D, R, r0, inter, dt, fused = case
    q, k = make(S, B, H, D, dt, 1, fused), make(S, B, Hk, D, dt, 2, fused)
    gq, gk = make(S, B, H, D, dt, 5, False), make(S, B, Hk, D, dt, 6, False)
    wq, wk = weights(D, 3)
    wq = wq if normed == "both" else None
    wk = None if normed == "none" else wk
    pos, f = positions(S, B, 4), inv(R)
    args = (on_gpu(q), on_gpu(k), gq.cuda(), gk.cuda(), f.cuda())
    kw = dict(positions=pos.cuda(), wq=on_gpu(wq), wk=on_gpu(wk), eps=EPS,
              rot_start=r0, interleaved=inter, rot_scale=1.25)
    got = dsa.dsa_norm_rope_bwd(*args, **kw)
    for name, x, w, g, dx, dw in (("q", q, wq, gq, got[0], got[2]),
                                  ("k", k, wk, gk, got[1], got[3])):
        rx, mx, rw, mw = norm_rope_bwd_ref(x, w, g, pos, f, r0, inter, EPS,
                                           1.25)
        assert_close("d" + name, dx, rx, mx, dt, 2.0 ** -17)
        assert (dw is None) == (w is None)
        if w is not None:
            err = (dw.double().cpu() - rw).abs()
            assert bool((err <= 2.0 ** -14 * mw + 1e-30).all())
    again = dsa.dsa_norm_rope_bwd(*args, **kw)
    for a, b in zip(got[:4], again[:4]):
        assert a is None or torch.equal(a, b)


@gpu
def test_without_keys_positions_or_rotation(dsa):
    q = make(9, 2, 3, 64, torch.bfloat16, 1, False)
    w, _ = weights(64, 2)
    f = inv(64)
    oq, ok = dsa.dsa_norm_rope_fwd(q.cuda(), None, f.cuda(), wq=w.cuda())
    assert ok is None
    pos = torch.arange(9)[:, None].expand(9, 2)
    want, mag = norm_rope_ref(q, w, pos, f, 0, False, EPS)
    assert_close("q", oq, want, mag, torch.bfloat16, 2.0 ** -19)
    oq, _ = dsa.dsa_norm_rope_fwd(q.cuda(), None, None)
    assert torch.equal(oq.cpu(), q)


@gpu
def test_zero_rows_and_special_values(dsa):
    """A row of zeros stays zero (eps under the root); a NaN or an infinity
    stays in its own row."""
    q = make(4, 1, 4, 64, torch.bfloat16, 1, False)
    q[0] = 0
    q[1, 0, 1, 3] = math.inf
    q[2, 0, 2, 5] = math.nan
    w, _ = weights(64, 2)
    f = inv(64)
    oq, _ = dsa.dsa_norm_rope_fwd(q.cuda(), None, f.cuda(), wq=w.cuda())
    oq = oq.cpu()
    assert bool((oq[0] == 0).all())
    clean = torch.ones(4, 1, 4, dtype=torch.bool)
    clean[1, 0, 1] = clean[2, 0, 2] = False
    assert bool(torch.isfinite(oq[clean]).all())
    want, mag = norm_rope_ref(q, w, torch.arange(4)[:, None], f, 0, False, EPS)
    assert_close("q", oq[clean], want[clean], mag[clean], torch.bfloat16,
                 2.0 ** -19)
    assert bool(torch.isnan(oq[2, 0, 2]).all())


def test_reference_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((3, 1, 2, 16), generator=g).double()
    w = (1 + 0.2 * torch.randn(16, generator=g)).double()
    gy = torch.randn((3, 1, 2, 16), generator=g).double()
    pos, f = torch.arange(3)[:, None] * 7, inv(8)

    def loss(x, w):
        return float((norm_rope_ref(x, w, pos, f, 4, True, EPS)[0] * gy).sum())
    dx, _, dw, _ = norm_rope_bwd_ref(x, w, gy, pos, f, 4, True, EPS)
    for _ in range(5):
        a, c = torch.randn(x.shape).double(), torch.randn(16).double()
        h = 1e-5
        num = (loss(x + h * a, w + h * c) - loss(x - h * a, w - h * c)) / (2 * h)
        ana = float((dx * a).sum() + (dw * c).sum())
        assert abs(num - ana) <= 1e-7 * (1 + abs(ana))


@gpu
def test_backward_against_differences(dsa):
    """Directional differences of the 64-bit forward against the kernel's
    gradient: off by no more than the elements' tolerances add up to."""
    g = torch.Generator().manual_seed(0)
    S, B, H, D = 6, 2, 3, 64
    x = torch.randn((S, B, H, D), generator=g)
    gy = torch.randn((S, B, H, D), generator=g)
    w, _ = weights(D, 1)
    pos, f = positions(S, B, 4), inv(D)
    dx, _, dw, _, _ = dsa.dsa_norm_rope_bwd(
        x.cuda(), None, gy.cuda(), None, f.cuda(), positions=pos.cuda(),
        wq=w.cuda(), eps=EPS)
    _, mx, _, mw = norm_rope_bwd_ref(x, w, gy, pos, f, 0, False, EPS)
    for _ in range(4):
        a = torch.randn(x.shape, generator=g).double()
        c = torch.randn(D, generator=g).double()
        h = 1e-5

        def loss(t):
            y = norm_rope_ref(x.double() + t * a, w.double() + t * c, pos, f,
                              0, False, EPS)[0]
            return float((y * gy.double()).sum())
        num = (loss(h) - loss(-h)) / (2 * h)
        ana = float((dx.double().cpu() * a).sum() + (dw.double().cpu() * c).sum())
        tol = float((2.0 ** -16 * mx * a.abs()).sum()
                    + (2.0 ** -14 * mw * c.abs()).sum()) + 1e-6 * abs(num)
        assert abs(num - ana) <= tol


# ---- paged append ------------------------------------------------------------

APPEND = [
    # S, B, H, Hk, D, R, r0, inter, page, pages, heads_first, with_q
    (1, 5, 8, 2, 128, 128, 0, False, 16, 8, False, True),
    (37, 3, 4, 4, 64, 32, 32, True, 64, 3, True, True),
    (9, 2, 0, 1, 96, 96, 0, False, 32, 4, False, False),
    (20, 2, 3, 3, 50, 10, 0, True, 7, 9, False, True),
]


@gpu
@pytest.mark.parametrize("case", APPEND)
def test_append(dsa, case):
    S, B, H, Hk, D, R, r0, inter, page, pages, heads_first, with_q = case
    bf = torch.bfloat16
    g = torch.Generator().manual_seed(7)
    total = H + 2 * Hk
    qkv = torch.randn((S, B, total * D), generator=g).to(bf)
    part = qkv.unflatten(-1, (total, D))
    q, k, v = part[:, :, :H], part[:, :, H:H + Hk], part[:, :, H + Hk:]
    P = B * pages + 3
    shape = (P, Hk, page, D) if heads_first else (P, page, Hk, D)
    kc = torch.randn(shape, generator=g).to(bf)
    vc = torch.randn(shape, generator=g).to(bf)
    table = torch.randperm(P, generator=g)[:B * pages].to(torch.int32).view(B, pages)
    first = torch.randint(0, page * pages - S + 1, (B,), generator=g)
    pos = (first[None, :] + torch.arange(S)[:, None]).to(torch.int32)
    pos[torch.rand((S, B), generator=g) < 0.2] = -1
    wq, wk = weights(D, 3)
    f = inv(R)
    gq = qkv.cuda().unflatten(-1, (total, D))
    gkc, gvc = kc.cuda(), vc.cuda()
    view = (lambda t: t.transpose(1, 2)) if heads_first else (lambda t: t)
    out_q, ws = dsa.dsa_paged_append(
        gq[:, :, H:H + Hk], gq[:, :, H + Hk:], view(gkc), view(gvc),
        table.cuda(), pos.cuda(), inv_freq=f.cuda(), wk=wk.cuda(), eps=EPS,
        rot_start=r0, interleaved=inter, q=gq[:, :, :H] if with_q else None,
        wq=wq.cuda() if with_q else None)
    assert dsa.dsa_indexer_check(ws) == 0
    want_k, mag_k = norm_rope_ref(k, wk, pos, f, r0, inter, EPS)
    got_k, got_v = view(gkc.cpu()), view(gvc.cpu())
    old_k, old_v = view(kc).clone(), view(vc).clone()
    for s in range(S):
        for b in range(B):
            p = int(pos[s, b])
            if p < 0:
                continue
            pg, off = int(table[b, p // page]), p % page
            assert_close("k", got_k[pg, off], want_k[s, b], mag_k[s, b], bf,
                         2.0 ** -19)
            assert torch.equal(got_v[pg, off], v[s, b])
            old_k[pg, off], old_v[pg, off] = got_k[pg, off], got_v[pg, off]
    # nothing else was touched
    assert torch.equal(old_k, got_k) and torch.equal(old_v, got_v)
    if with_q:
        want, mag = norm_rope_ref(q, wq, pos, f, r0, inter, EPS)
        assert_close("q", out_q, want, mag, bf, 2.0 ** -19)


@gpu
def test_append_reports_bad_pages(dsa):
    """Positions past the table and page ids outside the cache write nothing
    and are reported once."""
    bf = torch.bfloat16
    g = torch.Generator().manual_seed(7)
    k = torch.randn((1, 4, 2, 64), generator=g).to(bf).cuda()
    kc = torch.zeros((6, 8, 2, 64), dtype=bf, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.tensor([[0, 1], [6, 2], [-1, 3], [4, 5]], dtype=torch.int32)
    pos = torch.tensor([[3, 1, 2, 16]], dtype=torch.int32)
    _, ws = dsa.dsa_paged_append(k, k, kc, vc, table.cuda(), pos.cuda())
    assert dsa.dsa_indexer_check(ws) == 6
    assert dsa.dsa_indexer_check(ws) == 0
    assert torch.equal(kc[0, 3], k[0, 0])
    kc[0, 3] = 0
    assert not bool(kc.any())


@gpu
def test_append_past_32_bit_offsets(dsa):
    """A cache of more than 2^31 elements: the last page is written where it
    belongs."""
    bf = torch.bfloat16
    pages, page, Hk, D = 2 ** 31 // (64 * 8 * 128) + 2, 64, 8, 128
    kc = torch.zeros((pages, page, Hk, D), dtype=bf, device="cuda")
    k = torch.randn((1, 1, Hk, D), device="cuda").to(bf)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([[63]], dtype=torch.int32, device="cuda")
    _, ws = dsa.dsa_paged_append(k, k, kc, kc, table, pos)
    assert dsa.dsa_indexer_check(ws) == 0
    assert torch.equal(kc[-1, 63], k[0, 0])
    assert not bool(kc[:2].any())


@gpu
def test_other_stream_and_graph(dsa):
    """Work goes to the current stream, and the call can be captured."""
    q = make(40, 2, 8, 128, torch.bfloat16, 1, False).cuda()
    f = inv(128).cuda()
    want, _ = dsa.dsa_norm_rope_fwd(q, None, f)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got, _ = dsa.dsa_norm_rope_fwd(q, None, f)
    st.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_norm_rope_fwd(q, None, f, out_q=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# ---- frequencies and refusals (no GPU) ---------------------------------------

def test_inv_freq(dsa):
    f, m = dsa.rope_inv_freq(64, 10000.0)
    assert m == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, inv(64), rtol=1e-15, atol=0)
    lin, _ = dsa.rope_inv_freq(64, scaling=dict(type="linear", factor=4))
    assert torch.allclose(lin, f / 4, rtol=1e-15, atol=0)
    ntk, _ = dsa.rope_inv_freq(64, scaling=dict(type="ntk", factor=4))
    assert ntk[0] == 1 and math.isclose(ntk[-1], f[-1] / 4, rel_tol=1e-12)
    y, m = dsa.rope_inv_freq(64, scaling=dict(
        type="yarn", factor=8, original_max_position=4096))
    assert math.isclose(m, 0.1 * math.log(8) + 1)
    turns = 4096 * f / (2 * math.pi)
    assert torch.allclose(y[turns > 40], f[turns > 40], rtol=1e-15, atol=0)
    assert torch.allclose(y[turns < 0.7], f[turns < 0.7] / 8, rtol=1e-15, atol=0)
    assert bool(((y <= f) & (y >= f / 8)).all())
    for bad in (dict(type="linear", factor=0.5), dict(type="x", factor=2)):
        with pytest.raises(ValueError):
            dsa.rope_inv_freq(64, scaling=bad)
    with pytest.raises(ValueError):
        dsa.rope_inv_freq(7)


def test_calls_refuse_host_tensors(dsa):
    x = torch.zeros((2, 1, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((2, 8, 2, 64), dtype=torch.bfloat16)
    t = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dsa.dsa_norm_rope_fwd(x, x, inv(64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        dsa.dsa_norm_rope_bwd(x, x, x, x, inv(64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        dsa.dsa_paged_append(x, x, c, c, t, t)


FAKE = 1 << 20  # aligned, never read: every case fails before its use


def fwd_args(lib, **over):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, dtype=0, S=2, B=1, H=2, Hk=1,
             D=64, wq=None, wk=None, eps=1e-6, pos=None, inv=FAKE, r0=0, R=64,
             inter=0, m=1.0, oq=FAKE, ok=FAKE, st=None)
    a.update(over)
    return lib.dsa_norm_rope_fwd(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(oq=None), 1), (dict(ok=None), 1), (dict(S=0), 1),
    (dict(H=0), 1), (dict(Hk=0), 1), (dict(D=0), 1), (dict(R=63), 1),
    (dict(R=66), 1), (dict(r0=2), 1), (dict(r0=-1), 1), (dict(inv=None), 1),
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(m=0.0), 1),
    (dict(dtype=3), 2), (dict(D=258, R=64), 2), (dict(q=FAKE + 1), 1),
    (dict(inv=FAKE + 4), 1), (dict(S=1 << 30, B=4), 2),
])
def test_forward_refuses(dsa, over, code):
    assert fwd_args(dsa.load_library(), **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(gq=None), 1), (dict(gk=None), 1), (dict(dq=None), 1),
    (dict(wq=FAKE, gwq=None), 1), (dict(ws=None), 3), (dict(wsb=100), 3),
    (dict(ws=FAKE + 16), 1), (dict(D=300, R=64), 2),
])
def test_backward_refuses(dsa, over, code):
    a = dict(q=FAKE, qs=None, k=FAKE, ks=None, gq=FAKE, gk=FAKE, dtype=0, S=2,
             B=1, H=2, Hk=1, D=64, wq=None, wk=None, eps=1e-6, pos=None,
             inv=FAKE, r0=0, R=64, inter=0, m=1.0, dq=FAKE, dk=FAKE, gwq=None,
             gwk=None, ws=FAKE, wsb=1 << 30, st=None)
    a.update(over)
    assert dsa.load_library().dsa_norm_rope_bwd(*a.values()) == code


@pytest.mark.parametrize("over,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(kc=None), 1),
    (dict(table=None), 1), (dict(pos=None), 1), (dict(Hk=0), 1),
    (dict(q=FAKE, H=2), 1), (dict(pages=0), 1), (dict(page=0), 1),
    (dict(maxp=0), 1), (dict(ws=None), 3), (dict(wsb=255), 3),
    (dict(ws=FAKE + 16), 1), (dict(D=258), 2), (dict(table=FAKE + 2), 1),
])
def test_append_refuses(dsa, over, code):
    a = dict(k=FAKE, ks=None, v=FAKE, vs=None, q=None, qs=None, S=1, B=1, H=0,
             Hk=1, D=64, kc=FAKE, vc=FAKE, cs=None, pages=2, page=16,
             table=FAKE, maxp=2, pos=FAKE, wq=None, wk=None, eps=1e-6,
             inv=None, r0=0, R=0, inter=0, m=1.0, oq=None, ws=FAKE, wsb=256,
             st=None)
    a.update(over)
    assert dsa.load_library().dsa_paged_append(*a.values()) == code


@gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_no_rotation_whatever_shared_memory_holds(dsa, dt):
    """Without a rotation no angles are written; NaN that an earlier kernel
    left in shared memory stays out of the rows."""
    k = torch.full((640, 1, 1, 128), float("nan"), dtype=torch.bfloat16,
                   device="cuda")
    qa = torch.ones((640, 1, 64, 128), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((512, 3, 8, 128), dtype=torch.float32).to(dt).cuda()
    for _ in range(3):
        dsa.dsa_block_attn_fwd(qa, k, k, None, 64, 0.1, local_blocks=1)
        y, _ = dsa.dsa_norm_rope_fwd(x, None, None)
        assert torch.equal(y, x)
        dsa.dsa_block_attn_fwd(qa, k, k, None, 64, 0.1, local_blocks=1)
        g = dsa.dsa_norm_rope_bwd(x, None, x, None, None)[0]
        assert torch.equal(g, x)


@gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,H,Hk", [
    (64, 6, 2), (64, 4, 1), (128, 3, 1), (50, 5, 3), (256, 3, 1), (128, 4, 2)])
def test_backward_without_eps(dsa, dt, D, H, Hk):
    """eps = 0 is allowed, and heads that fill a warp's last group of rows in
    part leave nothing in the weights' gradients."""
    S, B = 3, 2
    q, k = make(S, B, H, D, dt, 1, False), make(S, B, Hk, D, dt, 2, False)
    gq, gk = make(S, B, H, D, dt, 5, False), make(S, B, Hk, D, dt, 6, False)
    wq, wk = weights(D, 3)
    pos, f = positions(S, B, 4), inv(D)
    got = dsa.dsa_norm_rope_bwd(
        q.cuda(), k.cuda(), gq.cuda(), gk.cuda(), f.cuda(),
        positions=pos.cuda(), wq=wq.cuda(), wk=wk.cuda(), eps=0.0)
    for name, x, w, g, dx, dw in (("q", q, wq, gq, got[0], got[2]),
                                  ("k", k, wk, gk, got[1], got[3])):
        rx, mx, rw, mw = norm_rope_bwd_ref(x, w, g, pos, f, 0, False, 0.0)
        assert_close("d" + name, dx, rx, mx, dt, 2.0 ** -17)
        err = (dw.double().cpu() - rw).abs()
        assert bool((err <= 2.0 ** -14 * mw + 1e-30).all()), "d weight " + name


@gpu
def test_errors_stay_in_a_workspace_of_their_own(dsa):
    """A bad page that the append reports outlives further appends and block
    attention in its workspace, and indexer calls in theirs; an indexer call in
    the same workspace begins with clearing the word, as the header says."""
    bf = torch.bfloat16
    k = torch.ones((1, 2, 2, 64), dtype=bf, device="cuda")
    kc = torch.zeros((4, 16, 2, 64), dtype=bf, device="cuda")
    good = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    bad = torch.tensor([[0, 1], [4, 3]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([[3, 5]], dtype=torch.int32, device="cuda")
    size = dsa.dsa_block_attn_workspace_size(1, 2, 2, 2, 64, 32, 16, 0, 1)
    ws = torch.zeros(max(size, 1 << 20), dtype=torch.uint8, device="cuda")
    index = lambda w: dsa.dsa_indexer_fwd(
        k, k[:, :, 0].contiguous(), torch.ones((1, 2, 2), device="cuda"), 1, 1,
        workspace=w)

    def step(index_ws):
        dsa.dsa_paged_append(k, k, kc, kc, bad, pos, workspace=ws)
        index(index_ws)
        dsa.dsa_paged_append(k, k, kc, kc, good, pos, workspace=ws)
        dsa.dsa_block_attn_paged_fwd(k, kc, kc, good, None, 16, 0.1,
                                     q_pos=pos[0], local_blocks=1,
                                     workspace=ws)
    step(torch.empty_like(ws))
    assert dsa.dsa_indexer_check(ws) == 6
    assert dsa.dsa_indexer_check(ws) == 0
    step(ws)
    assert dsa.dsa_indexer_check(ws) == 0
