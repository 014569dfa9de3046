"""Cases, plain forms and 64-bit definitions of the operators around block
sparse attention: the per-head norm with the rotation of positions, the append
to a paged cache, and attention over selected blocks (training, prefill from a
paged cache, single tokens).

`own` chooses between the plain torch forms and the framework's kernels.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the queries and keys of one decoding step, too small to fill the GPU
        dict(name="norm_rope_step", op="norm_rope", S=1, B=64, H=32, Hk=8,
             D=128, R=128, r0=0, inter=False, dtype="fp16", fused=False,
             base=1e4, pos0=8000, weights=True),
        # a long prefill, read in place out of a fused projection's output;
        # half of the head rotated, in pairs of neighbours
        dict(name="norm_rope_prefill", op="norm_rope", S=32768, B=1, H=64,
             Hk=8, D=128, R=64, r0=64, inter=True, dtype="bf16", fused=True,
             base=5e5, pos0=0, weights=True),
        # the gradient of the same for a training batch
        dict(name="norm_rope_grad", op="norm_rope_bwd", S=4096, B=2, H=32,
             Hk=8, D=128, R=128, r0=0, inter=False, dtype="bf16", fused=True,
             base=1e4, pos0=0, weights=True),
        # one token of each of 64 sequences into the cache
        dict(name="append_step", op="append", S=1, B=64, H=64, Hk=4, D=128,
             R=128, r0=0, inter=False, page=64, pages=32, base=5e5,
             pad=0.05, weights=True),
        # a chunk of a long prompt, a ragged batch with padded rows
        dict(name="append_chunk", op="append", S=2048, B=4, H=40, Hk=8, D=64,
             R=32, r0=0, inter=False, page=128, pages=64, base=1e4,
             pad=0.1, weights=True),
        # training step at the V3.2-style prefill's length
        dict(name="attn_train_4k", op="attn_train", S=4096, B=1, H=64, Hk=4,
             D=128, block=64, topk=16, local=1, shared=False, hold=32,
             q_pos=False),
        # odd lengths, small blocks, twelve heads a group, every query its own
        # selection (nothing shared between neighbours)
        dict(name="attn_train_odd", op="attn_train", S=2047, B=2, H=24, Hk=2,
             D=64, block=32, topk=24, local=1, shared=False, hold=1,
             q_pos=False),
        # prefill at the C4 workload's length, one selection for all heads
        dict(name="attn_prefill_16k", op="attn_fwd", S=16384, B=1, H=64,
             Hk=8, D=128, block=64, topk=16, local=2, shared=True, hold=32,
             q_pos=False),
        # a chunk of a prompt against the pages before it; five heads a group
        dict(name="attn_chunk_paged", op="attn_paged", S=777, B=3, H=40, Hk=8,
             D=64, block=64, topk=32, local=2, shared=False, hold=16,
             page=128, pos_lo=9000, pos_hi=20000),
        # one token of one sequence: latency
        dict(name="attn_step_1", op="attn_paged", S=1, B=1, H=32, Hk=8,
             D=128, block=64, topk=16, local=1, shared=False, hold=1, page=64,
             pos_lo=8000, pos_hi=8191),
        # one token of 64 sequences, the decode workload's lengths
        dict(name="attn_step_64", op="attn_paged", S=1, B=64, H=64, Hk=4,
             D=128, block=64, topk=32, local=2, shared=True, hold=1, page=64,
             pos_lo=2048, pos_hi=32767),
        # four draft tokens of eight sequences, small blocks
        dict(name="attn_draft_8", op="attn_paged", S=4, B=8, H=32, Hk=4,
             D=128, block=16, topk=64, local=4, shared=False, hold=2, page=64,
             pos_lo=1000, pos_hi=16000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "attn_fwd",
                     "attn_train", "attn_train", "attn_paged", "attn_paged"])
    if op in ("norm_rope", "norm_rope_bwd", "append"):
        D = rng.choice([64, 96, 128, 128, 192, 256])
        R = rng.choice([D, D // 2, 32])
        r0 = rng.choice([0, D - R])
        Hk = rng.choice([1, 2, 4, 8])
        H = Hk * rng.choice([1, 3, 4, 8, 16])
        B = rng.randint(1, 5)
        case = dict(op=op, B=B, H=H, Hk=Hk, D=D, R=R, r0=r0,
                    inter=rng.random() < 0.5, base=rng.choice([1e4, 5e5]),
                    weights=rng.random() < 0.8)
        cap = max(1, (1 << 27) // ((H + Hk) * D * B))
        if op == "append":
            case["page"] = rng.choice([16, 64, 128, 256])
            case["pages"] = rng.randint(8, 32)
            room = case["page"] * case["pages"] - 1
            case["S"] = _log(rng, 1, min(4096, cap, room))
            case["pad"] = rng.choice([0.0, 0.1, 0.5])
        else:
            case["S"] = _log(rng, 1, min(16384, cap))
            case["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
            case["fused"] = rng.random() < 0.5
            case["pos0"] = rng.choice([0, 0, 1000, 100000, 1000000])
        return case
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 4, 5, 8, 8, 12, 16])
    case = dict(op=op, B=rng.randint(1, 3), H=Hk * G, Hk=Hk,
                D=rng.choice([64, 128]), block=rng.choice([16, 32, 64, 128]),
                local=rng.choice([1, 2]), shared=rng.random() < 0.4,
                hold=rng.choice([1, 8, 32]))
    case["topk"] = max(1, rng.choice([128, 512, 1024]) // case["block"])
    if op == "attn_paged":
        case["S"] = rng.choice([1, 1, 2, 5, 64, 333])
        case["B"] = rng.randint(1, 24) if case["S"] < 8 else rng.randint(1, 3)
        case["page"] = case["block"] * rng.choice([1, 2, 4])
        case["pos_lo"] = _log(rng, 16, 4000)
        case["pos_hi"] = case["pos_lo"] + _log(rng, 16, 16000)
    else:
        top = 4096 if op == "attn_train" else 8192
        rows = (1 << 18) // (case["B"] * case["H"])
        case["S"] = _log(rng, 1, max(2, min(top, rows)))
        case["q_pos"] = op == "attn_fwd" and rng.random() < 0.5
    return case


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype=torch.float32, scale=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x * scale).to(dtype)


def _inv_freq(case):
    i = torch.arange(case["R"] // 2, dtype=torch.float64, device="cuda")
    return case["base"] ** (-2.0 * i / case["R"])


def _weights(g, case):
    if not case["weights"]:
        return None, None
    D = case["D"]
    return (1 + _randn(g, (D,), scale=0.2), 1 + _randn(g, (D,), scale=0.2))


def _select(g, case, pos, nblk):
    """Block ids [B, S, Hs, topk]: the best older blocks of a smooth random
    score, in descending order, -1 where there are fewer; the score's query
    side changes every `hold` queries, as neighbouring queries ask for much
    the same blocks.  The first block scores highest (an attention sink)."""
    B, S = pos.shape
    Hs = 1 if case["shared"] else case["Hk"]
    n, hold = case["topk"], case["hold"]
    own_blk = pos // case["block"]
    older = own_blk - case["local"] + 1            # blocks before the local ones
    ids = torch.arange(nblk, device="cuda")
    out = torch.full((B, S, Hs, n), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        for h in range(Hs):
            bf = _randn(g, (8, nblk))
            qf = _randn(g, ((S + hold - 1) // hold, 8))
            qf = qf.repeat_interleave(hold, dim=0)[:S]
            qf = qf + 0.25 * _randn(g, (S, 8))
            score = qf @ bf
            score[:, 0] = 1e9
            score.masked_fill_(ids[None, :] >= older[b][:, None], -math.inf)
            v, i = torch.topk(score, min(n, nblk), dim=1)
            out[b, :, h, :v.shape[1]] = torch.where(
                v > -math.inf, i, -1).to(torch.int32)
    return out[:, :, 0].contiguous() if case["shared"] else out


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    S, B, H, Hk, D = (case[x] for x in ("S", "B", "H", "Hk", "D"))
    st = dict(case=case)
    bf = torch.bfloat16
    if op in ("norm_rope", "norm_rope_bwd"):
        dt = _DT[case["dtype"]]
        if case["fused"]:
            qkv = _randn(g, (S, B, (H + 2 * Hk) * D), dt)
            st["q"] = qkv[..., :H * D].view(S, B, H, D)
            st["k"] = qkv[..., H * D:(H + Hk) * D].view(S, B, Hk, D)
        else:
            st["q"] = _randn(g, (S, B, H, D), dt)
            st["k"] = _randn(g, (S, B, Hk, D), dt)
        first = torch.randint(0, 64, (B,), generator=g, device="cuda")
        st["pos"] = (case["pos0"] + first[None, :]
                     + torch.arange(S, device="cuda")[:, None]).to(torch.int32)
        st["inv_freq"] = _inv_freq(case)
        st["wq"], st["wk"] = _weights(g, case)
        if op == "norm_rope_bwd":
            st["gq"] = _randn(g, (S, B, H, D), dt)
            st["gk"] = _randn(g, (S, B, Hk, D), dt)
        return st
    if op == "append":
        page, pages = case["page"], case["pages"]
        qkv = _randn(g, (S, B, (H + 2 * Hk) * D), bf)
        st["q"] = qkv[..., :H * D].view(S, B, H, D)
        st["k"] = qkv[..., H * D:(H + Hk) * D].view(S, B, Hk, D)
        st["v"] = qkv[..., (H + Hk) * D:].view(S, B, Hk, D)
        st["k_cache"] = _randn(g, (B * pages, page, Hk, D), bf)
        st["v_cache"] = _randn(g, (B * pages, page, Hk, D), bf)
        st["table"] = torch.randperm(B * pages, generator=g, device="cuda"
                                     ).to(torch.int32).view(B, pages)
        first = torch.randint(0, page * pages - S, (B,), generator=g,
                              device="cuda")
        pos = first[None, :] + torch.arange(S, device="cuda")[:, None]
        padded = torch.rand((S, B), generator=g, device="cuda") < case["pad"]
        st["pos"] = torch.where(padded, -1, pos).to(torch.int32)
        st["inv_freq"] = _inv_freq(case)
        st["wq"], st["wk"] = _weights(g, case)
        if own:
            st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return st
    st["scale"] = D ** -0.5
    st["q"] = _randn(g, (S, B, H, D), bf)
    if op == "attn_paged":
        page, block = case["page"], case["block"]
        q_pos = torch.randint(case["pos_lo"], case["pos_hi"] + 1, (B,),
                              generator=g, device="cuda")
        T = case["pos_hi"] + S
        pages = -(-T // page)
        st["k_cache"] = torch.randn((B * pages, page, Hk, D), generator=g,
                                    device="cuda", dtype=bf)
        st["v_cache"] = torch.randn((B * pages, page, Hk, D), generator=g,
                                    device="cuda", dtype=bf)
        st["table"] = torch.randperm(B * pages, generator=g, device="cuda"
                                     ).to(torch.int32).view(B, pages)
        nblk = pages * page // block
    else:
        off = 64 * 7 + 13 if case["q_pos"] else 0
        T = S + off
        q_pos = torch.full((B,), off, device="cuda")
        st["k"] = _randn(g, (T, B, Hk, D), bf)
        st["v"] = _randn(g, (T, B, Hk, D), bf)
        nblk = -(-T // case["block"])
    pos = q_pos[:, None] + torch.arange(S, device="cuda")[None, :]
    st["blocks"] = _select(g, case, pos, nblk)
    st["q_pos"] = q_pos.to(torch.int32)
    if op == "attn_train":
        st["go"] = _randn(g, (S, B, H, D), bf)
    if own:
        # the workspaces that a program keeps from step to step
        import dsa_sparse_attention_fwd_gb300 as dsa
        shape = (S, B, H, Hk, D, nblk * case["block"], case["block"],
                 case["topk"], case["local"])
        sizes = {"ws": dsa.dsa_block_attn_workspace_size(*shape)}
        if op == "attn_train":
            sizes["ws_bwd"] = dsa.dsa_block_attn_bwd_workspace_size(*shape)
        for name, size in sizes.items():
            st[name] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    return st


# --------------------------------------------------------------------------
# plain forms: 32 bits, elementary operations
# --------------------------------------------------------------------------

def _cos_sin(pos, inv_freq):
    # far positions: the angle in 64 bits
    a = pos.to(torch.float64)[..., None] * inv_freq
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, case, back=False):
    """x [S,B,H,D] fp32, cos/sin [S,B,R/2]."""
    r0, R = case["r0"], case["R"]
    c, s = cos[:, :, None, :], sin[:, :, None, :]
    if back:
        s = -s
    part = x[..., r0:r0 + R]
    if case["inter"]:
        a, b = part[..., 0::2], part[..., 1::2]
        y = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    else:
        a, b = part[..., :R // 2], part[..., R // 2:]
        y = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    return torch.cat([x[..., :r0], y, x[..., r0 + R:]], dim=-1)


def _plain_norm_rope(x, w, cos, sin, case):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
    return _rotate(y, cos, sin, case).to(x.dtype)


def _plain_norm_rope_bwd(x, w, gy, cos, sin, case):
    u = _rotate(gy.float(), cos, sin, case, back=True)
    if w is None:
        return u.to(x.dtype), None
    xf = x.float()
    rstd = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6)
    xh = xf * rstd
    gw = (u * xh).sum((0, 1, 2))
    u = u * w
    gx = rstd * (u - xh * (u * xh).mean(-1, keepdim=True))
    return gx.to(x.dtype), gw


def _plain_append(st):
    case = st["case"]
    cos, sin = _cos_sin(st["pos"], st["inv_freq"])
    q = _plain_norm_rope(st["q"], st["wq"], cos, sin, case)
    k = _plain_norm_rope(st["k"], st["wk"], cos, sin, case)
    pos = st["pos"].long()
    keep = pos >= 0
    page = case["page"]
    b = torch.arange(case["B"], device="cuda")[None, :].expand_as(pos)
    pg = st["table"].long()[b[keep], pos[keep] // page]
    st["k_cache"][pg, pos[keep] % page] = k[keep]
    st["v_cache"][pg, pos[keep] % page] = st["v"][keep]
    return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _ids(st, s0, s1):
    """Block ids of rows s0..s1 of every sequence with the local blocks, each
    block once: [B, C, Hs, n + local], -1 where empty; and positions [B, C]."""
    case = st["case"]
    pos = st["q_pos"].long()[:, None] + torch.arange(s0, s1, device="cuda")
    bl = st["blocks"][:, s0:s1].long()
    if case["shared"]:
        bl = bl[:, :, None]
    own_blk = pos // case["block"]
    loc = own_blk[..., None] - torch.arange(case["local"], device="cuda")
    loc = loc[:, :, None].expand(*bl.shape[:3], case["local"])
    ids = torch.cat([bl, loc], -1).sort(-1).values
    again = torch.zeros_like(ids, dtype=torch.bool)
    again[..., 1:] = ids[..., 1:] == ids[..., :-1]
    return torch.where(again | (ids < 0), -1, ids), pos


def _gather(st, b, ids, pos):
    """Token numbers [C, Hk, m] and their visibility for one sequence."""
    case = st["case"]
    blk = case["block"]
    j = (ids[..., None] * blk + torch.arange(blk, device="cuda")).flatten(-2)
    ok = (ids[..., None] >= 0).expand(*ids.shape, blk).flatten(-2)
    ok = ok & (j <= pos[:, None, None])
    return (torch.where(ok, j, 0).expand(-1, case["Hk"], -1),
            ok.expand(-1, case["Hk"], -1))


def _kv_rows(st, b, j):
    """fp32 keys and values [C, Hk, m, D] of the tokens j [C, Hk, m]."""
    h = torch.arange(st["case"]["Hk"], device="cuda")[None, :, None]
    if "table" in st:
        page = st["case"]["page"]
        pg, off = st["table"].long()[b][j // page], j % page
        return st["k_cache"][pg, off, h].float(), st["v_cache"][pg, off, h].float()
    return st["k"][j, b, h].float(), st["v"][j, b, h].float()


def _chunks(case):
    m = (case["topk"] + case["local"]) * case["block"]
    step = max(1, (1 << 27) // (m * case["Hk"] * case["D"]))
    return [(s, min(case["S"], s + step)) for s in range(0, case["S"], step)]


def _probs(st, b, s0, s1):
    case = st["case"]
    C, Hk, D = s1 - s0, case["Hk"], case["D"]
    ids, pos = _ids(st, s0, s1)
    j, ok = _gather(st, b, ids[b], pos[b])
    kf, vf = _kv_rows(st, b, j)
    q = st["q"][s0:s1, b].float().view(C, Hk, case["H"] // Hk, D)
    x = torch.matmul(q, kf.transpose(-1, -2)) * st["scale"]
    x = x.masked_fill(~ok[:, :, None, :], -math.inf)
    mx = x.amax(-1, keepdim=True)
    mx = torch.where(mx > -math.inf, mx, 0.0)
    e = torch.exp(x - mx)
    l = e.sum(-1, keepdim=True)
    p = torch.where(l > 0, e / l, 0.0)
    return q, kf, vf, j, p, (mx + torch.log(l))[..., 0]


def _plain_attn(st):
    case = st["case"]
    S, B, H, D = (case[x] for x in "SBHD")
    o = torch.empty((S, B, H, D), device="cuda", dtype=torch.bfloat16)
    lse = torch.empty((S, B, H), device="cuda")
    for b in range(B):
        for s0, s1 in _chunks(case):
            _, _, vf, _, p, ls = _probs(st, b, s0, s1)
            o[s0:s1, b] = torch.matmul(p, vf).flatten(1, 2).to(o.dtype)
            lse[s0:s1, b] = ls.flatten(1)
    return {"o": o, "lse": lse}


def _plain_attn_train(st):
    case = st["case"]
    S, B, H, D, Hk = (case[x] for x in ("S", "B", "H", "D", "Hk"))
    T = st["k"].shape[0]
    out = _plain_attn(st)
    gq = torch.empty((S, B, H, D), device="cuda", dtype=torch.bfloat16)
    gk = torch.zeros((B, T * Hk, D), device="cuda")
    gv = torch.zeros((B, T * Hk, D), device="cuda")
    for b in range(B):
        for s0, s1 in _chunks(case):
            q, kf, vf, j, p, _ = _probs(st, b, s0, s1)
            go = st["go"][s0:s1, b].float().view(q.shape)
            o = torch.matmul(p, vf)
            dp = torch.matmul(go, vf.transpose(-1, -2))
            ds = p * (dp - (go * o).sum(-1, keepdim=True)) * st["scale"]
            gq[s0:s1, b] = torch.matmul(ds, kf).flatten(1, 2).to(gq.dtype)
            at = (j * Hk + torch.arange(Hk, device="cuda")[None, :, None]).flatten()
            gv[b].index_add_(0, at, torch.matmul(p.transpose(-1, -2), go).view(-1, D))
            gk[b].index_add_(0, at, torch.matmul(ds.transpose(-1, -2), q).view(-1, D))
    out["gq"] = gq
    for name, t in (("gk", gk), ("gv", gv)):
        out[name] = t.view(B, T, Hk, D).transpose(0, 1).to(torch.bfloat16)
    return out


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "append":
        return _plain_append(st)
    if op in ("attn_fwd", "attn_paged"):
        return _plain_attn(st)
    if op == "attn_train":
        return _plain_attn_train(st)
    cos, sin = _cos_sin(st["pos"], st["inv_freq"])
    if op == "norm_rope":
        return {"q": _plain_norm_rope(st["q"], st["wq"], cos, sin, case),
                "k": _plain_norm_rope(st["k"], st["wk"], cos, sin, case)}
    gq, gwq = _plain_norm_rope_bwd(st["q"], st["wq"], st["gq"], cos, sin, case)
    gk, gwk = _plain_norm_rope_bwd(st["k"], st["wk"], st["gk"], cos, sin, case)
    out = {"gq": gq, "gk": gk}
    if gwq is not None:
        out.update(gwq=gwq, gwk=gwk)
    return out


# --------------------------------------------------------------------------
# the framework's kernels
# --------------------------------------------------------------------------

def _own(st):
    import dsa_sparse_attention_fwd_gb300 as dsa
    case = st["case"]
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd", "append"):
        rope = dict(eps=1e-6, rot_start=case["r0"], interleaved=case["inter"])
    if op == "norm_rope":
        q, k = dsa.dsa_norm_rope_fwd(
            st["q"], st["k"], st["inv_freq"], positions=st["pos"],
            wq=st["wq"], wk=st["wk"], **rope)
        return {"q": q, "k": k}
    if op == "norm_rope_bwd":
        gq, gk, gwq, gwk, _ = dsa.dsa_norm_rope_bwd(
            st["q"], st["k"], st["gq"], st["gk"], st["inv_freq"],
            positions=st["pos"], wq=st["wq"], wk=st["wk"], **rope)
        out = {"gq": gq, "gk": gk}
        if gwq is not None:
            out.update(gwq=gwq, gwk=gwk)
        return out
    if op == "append":
        q, _ = dsa.dsa_paged_append(
            st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"],
            st["pos"], inv_freq=st["inv_freq"], wk=st["wk"], q=st["q"],
            wq=st["wq"], workspace=st["ws"], **rope)
        return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    args = dict(block_size=case["block"], scale=st["scale"],
                q_pos=st["q_pos"], local_blocks=case["local"])
    if op == "attn_paged":
        o, lse, _ = dsa.dsa_block_attn_paged_fwd(
            st["q"], st["k_cache"], st["v_cache"], st["table"], st["blocks"],
            workspace=st["ws"], **args)
        return {"o": o, "lse": lse}
    o, lse, _ = dsa.dsa_block_attn_fwd(st["q"], st["k"], st["v"],
                                       st["blocks"], workspace=st["ws"],
                                       **args)
    out = {"o": o, "lse": lse}
    if op == "attn_train":
        gq, gk, gv, _ = dsa.dsa_block_attn_bwd(
            st["q"], st["k"], st["v"], o, lse, st["go"], st["blocks"],
            workspace=st["ws_bwd"], **args)
        out.update(gq=gq, gk=gk, gv=gv)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def _attended(case):
    """Keys that the rows of one sequence and head attend to (positions of
    the paged cases at the middle of their range)."""
    if case["op"] == "attn_paged":
        p0 = (case["pos_lo"] + case["pos_hi"]) // 2
    else:
        p0 = 64 * 7 + 13 if case["q_pos"] else 0
    pos = p0 + np.arange(case["S"], dtype=np.int64)
    blk = case["block"]
    own_blk = pos // blk
    loc = np.minimum(case["local"], own_blk + 1)
    older = np.minimum(case["topk"], own_blk + 1 - loc)
    return int(((older + loc - 1) * blk + pos % blk + 1).sum()), int(pos[-1]) + 1


def work(case):
    S, B, H, Hk, D = (case[x] for x in ("S", "B", "H", "Hk", "D"))
    op = case["op"]
    rows = S * B
    if op in ("norm_rope", "norm_rope_bwd"):
        el = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        n = rows * (H + Hk) * D
        if op == "norm_rope":
            return {"bytes": 2 * n * el + 4 * rows, "flops": 8 * n}
        return {"bytes": 3 * n * el + 4 * rows, "flops": 20 * n}
    if op == "append":
        kept = int(round(rows * (1 - case["pad"])))
        n = 2 * rows * H * D + 4 * kept * Hk * D
        return {"bytes": 2 * n + 8 * rows, "flops": 8 * (rows * H + kept * Hk) * D}
    keys, T = _attended(case)
    Hs = 1 if case["shared"] else Hk
    once = min(keys, T)     # tokens of one sequence that have to be read
    kv = 2 * B * once * Hk * D * 2
    q = rows * H * D * 2
    flops = 4 * B * keys * H * D
    by = 2 * q + kv + rows * H * 4 + 4 * rows * Hs * case["topk"]
    if op == "attn_train":
        # the backward reads q, k, v, o, its gradient and the ids, and writes
        # three gradients; five products
        by += 4 * q + 2 * kv + rows * H * 4 + 4 * rows * Hs * case["topk"]
        flops += 10 * B * keys * H * D
    return {"bytes": by, "flops": flops}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def _exact_norm_rope(x, w, pos, case):
    """x [S,B,H,D] fp64 -> fp64, differentiable; the rotation as a complex
    product."""
    R, r0 = case["R"], case["r0"]
    if w is not None:
        ms = x.square().mean(dim=3, keepdim=True)
        x = x / torch.sqrt(ms + 1e-6) * w.double()
    lo, part, hi = x.split([r0, R, case["D"] - r0 - R], dim=3)
    theta = torch.outer(pos.double().flatten(), _inv_freq(case))
    turn = torch.polar(torch.ones_like(theta), theta)
    turn = turn.view(*pos.shape, 1, R // 2)
    if case["inter"]:
        z = torch.view_as_complex(part.reshape(*part.shape[:3], R // 2, 2).contiguous())
        y = torch.view_as_real(z * turn).reshape(part.shape)
    else:
        z = torch.complex(part[..., :R // 2], part[..., R // 2:]) * turn
        y = torch.cat([z.real, z.imag], dim=3)
    return torch.cat([lo, y, hi], dim=3)


def _exact_small(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        return {x: _exact_norm_rope(st[x].double(), st["w" + x], st["pos"], case)
                for x in "qk"}
    if op == "append":
        q, k = (_exact_norm_rope(st[x].double(), st["w" + x], st["pos"], case)
                for x in "qk")
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        flat_k, flat_v = kc.flatten(0, 1), vc.flatten(0, 1)
        for b in range(case["B"]):
            p = st["pos"][:, b].long()
            rows = torch.nonzero(p >= 0)[:, 0]
            p = p[rows]
            slot = st["table"][b].long()[p // case["page"]] * case["page"] + p % case["page"]
            flat_k[slot] = k[rows, b]
            flat_v[slot] = st["v"][rows, b].double()
        return {"q": q, "k_cache": kc, "v_cache": vc}
    out = {}
    for x in "qk":
        a = st[x].double().requires_grad_(True)
        w = st["w" + x]
        wd = None if w is None else w.double().requires_grad_(True)
        y = _exact_norm_rope(a, wd, st["pos"], case)
        leaves = [a] if w is None else [a, wd]
        grads = torch.autograd.grad(y, leaves, st["g" + x].double())
        out["g" + x] = grads[0]
        if w is not None:
            out["gw" + x] = grads[1]
    return out


def _exact_attn(case, seed):
    """Block by block: each block of keys meets the rows that hold it."""
    st = prepare(case, seed)
    S, B, H, Hk, D = (case[x] for x in ("S", "B", "H", "Hk", "D"))
    G, blk = H // Hk, case["block"]
    train = case["op"] == "attn_train"
    f64 = dict(dtype=torch.float64, device="cuda")
    o = torch.zeros((S, B, H, D), **f64)
    lse = torch.full((S, B, H), -math.inf, **f64)
    paged = "table" in st
    T = st["table"].shape[1] * case["page"] if paged else st["k"].shape[0]
    if train:
        gq = torch.zeros((S, B, H, D), **f64)
        gk = torch.zeros((T, B, Hk, D), **f64)
        gv = torch.zeros((T, B, Hk, D), **f64)
    nblk = -(-T // blk)
    for b in range(B):
        pos = int(st["q_pos"][b]) + torch.arange(S, device="cuda")
        if paged:
            kb = st["k_cache"][st["table"][b].long()].flatten(0, 1)
            vb = st["v_cache"][st["table"][b].long()].flatten(0, 1)
        else:
            kb, vb = st["k"][:, b], st["v"][:, b]
        for hk in range(Hk):
            chosen = st["blocks"][b] if case["shared"] else st["blocks"][b, :, hk]
            holds = torch.zeros((S, nblk + 1), dtype=torch.bool, device="cuda")
            holds.scatter_(1, torch.where(chosen >= 0, chosen, nblk).long(), True)
            holds = holds[:, :nblk]
            gap = (pos // blk)[:, None] - torch.arange(nblk, device="cuda")[None, :]
            holds = (holds | (gap < case["local"])) & (gap >= 0)
            pairs = torch.nonzero(holds.t())           # by block, then row
            counts = torch.bincount(pairs[:, 0], minlength=nblk).tolist()
            row_sets = torch.split(pairs[:, 1], counts)
            heads = slice(hk * G, hk * G + G)
            q = st["q"][:, b, heads].double()
            m = torch.full((S, G), -math.inf, **f64)
            l = torch.zeros((S, G), **f64)
            acc = torch.zeros((S, G, D), **f64)

            def logits(n, rows):
                t1 = min(T, n * blk + blk)
                x = torch.einsum("rgd,td->rgt", q[rows], kb[n * blk:t1, hk].double())
                t = torch.arange(n * blk, t1, device="cuda")
                x = torch.where(t[None, None, :] <= pos[rows][:, None, None],
                                x * st["scale"], -math.inf)
                return x, vb[n * blk:t1, hk].double(), t1

            for n, rows in enumerate(row_sets):
                if counts[n] == 0:
                    continue
                x, v, _ = logits(n, rows)
                top = torch.maximum(m[rows], x.amax(2))
                old = torch.exp(m[rows] - top)
                e = torch.exp(x - top[..., None])
                l[rows] = l[rows] * old + e.sum(2)
                acc[rows] = acc[rows] * old[..., None] + torch.einsum("rgt,td->rgd", e, v)
                m[rows] = top
            some = l > 0
            o[:, b, heads] = torch.where(some[..., None], acc / l[..., None], 0.0)
            lse[:, b, heads] = torch.where(some, m + torch.log(l), -math.inf)
            if not train:
                continue
            go = st["go"][:, b, heads].double()
            delta = (go * o[:, b, heads]).sum(2)
            for n, rows in enumerate(row_sets):
                if counts[n] == 0:
                    continue
                x, v, t1 = logits(n, rows)
                p = torch.exp(x - lse[:, b, heads][rows][..., None])
                dp = torch.einsum("rgd,td->rgt", go[rows], v)
                ds = p * (dp - delta[rows][..., None]) * st["scale"]
                kk = kb[n * blk:t1, hk].double()
                gq[:, b, heads].index_add_(0, rows, torch.einsum("rgt,td->rgd", ds, kk))
                gk[n * blk:t1, b, hk] = torch.einsum("rgt,rgd->td", ds, q[rows])
                gv[n * blk:t1, b, hk] = torch.einsum("rgt,rgd->td", p, go[rows])
    out = {"o": o, "lse": lse}
    if train:
        out.update(gq=gq, gk=gk, gv=gv)
    return out


def exact(case, seed):
    if case["op"].startswith("attn"):
        return _exact_attn(case, seed)
    return _exact_small(case, seed)
