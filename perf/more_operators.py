"""Cases, plain forms and 64-bit definitions of the operators of a paged cache
held in 8 bits: the append that quantises (after the norm and the rotation of
the keys), the read back, and attention over it, of selected blocks of keys or
of all keys.

A cache holds e4m3 values [pages, page, Hk, D] and one power of two for each
`group` of consecutive tokens and head [pages, page / group, Hk]: a key or
value is its 8-bit value times the group's scale.

`own` chooses between the plain torch forms and the framework's kernels.
"""
from __future__ import annotations

import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
TOP = 448.0          # the largest e4m3 value
MIN_EXP, MAX_EXP = -40, 40   # of a scale


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one decoding step of 64 sequences, too small to fill the GPU; most
        # tokens join a group that has tokens already
        dict(name="append_step", op="append", S=1, B=64, H=64, Hk=4, D=128,
             R=128, r0=0, inter=False, page=64, pages=32, group=64, base=5e5,
             ragged=False, turned=False),
        # a chunk of a long prompt out of a fused projection's output, a
        # ragged batch; half of the head rotated
        dict(name="append_chunk", op="append", S=2048, B=4, H=40, Hk=8, D=64,
             R=32, r0=0, inter=False, page=128, pages=64, group=128, base=1e4,
             ragged=True, turned=False),
        # keys that are turned already, small groups, odd lengths
        dict(name="append_turned", op="append", S=333, B=3, H=0, Hk=6, D=96,
             R=0, r0=0, inter=False, page=80, pages=24, group=16, base=1e4,
             ragged=True, turned=True),
        # two long prefixes read back for a dense product
        dict(name="read_prefix", op="read", T=30000, B=2, Hk=8, D=128,
             page=64, pages=480, group=64, pos_lo=20000, pos_hi=30000),
        # a ragged batch of short ones, from the middle of their pages
        dict(name="read_short", op="read", T=777, B=5, Hk=4, D=64, page=128,
             pages=10, group=32, pos_lo=3, pos_hi=777),
        # one token of one sequence over its selected blocks: latency
        dict(name="attn_step_1", op="attn", S=1, B=1, H=32, Hk=8, D=128,
             block=64, topk=16, local=1, shared=False, hold=1, page=64,
             group=64, pos_lo=8000, pos_hi=8191),
        # one token of 64 sequences over their selected blocks
        dict(name="attn_step_64", op="attn", S=1, B=64, H=64, Hk=4, D=128,
             block=64, topk=32, local=2, shared=True, hold=1, page=64,
             group=64, pos_lo=2048, pos_hi=32767),
        # one token of one sequence over all of a long cache
        dict(name="attn_all_1", op="attn", S=1, B=1, H=32, Hk=8, D=128,
             block=128, topk=0, local=0, shared=True, hold=1, page=128,
             group=128, pos_lo=131000, pos_hi=131071),
        # one token of 64 sequences of many lengths over all their keys
        dict(name="attn_all_64", op="attn", S=1, B=64, H=64, Hk=4, D=128,
             block=64, topk=0, local=0, shared=True, hold=1, page=64,
             group=64, pos_lo=2048, pos_hi=32767),
        # four draft tokens of eight sequences, small blocks
        dict(name="attn_draft_8", op="attn", S=4, B=8, H=32, Hk=4, D=128,
             block=16, topk=64, local=4, shared=False, hold=2, page=64,
             group=32, pos_lo=1000, pos_hi=16000),
        # a chunk of a prompt against the pages before it; five heads a group
        dict(name="attn_chunk", op="attn", S=777, B=3, H=40, Hk=8, D=64,
             block=64, topk=32, local=2, shared=False, hold=16, page=128,
             group=64, pos_lo=9000, pos_hi=20000),
        # a chunk against all keys before it (a layer without a selection)
        dict(name="attn_chunk_all", op="attn", S=512, B=2, H=32, Hk=8, D=128,
             block=64, topk=0, local=0, shared=True, hold=1, page=64,
             group=64, pos_lo=8000, pos_hi=15800),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attn", "attn", "attn"])
    group = rng.choice([16, 32, 64, 128])
    if op == "append":
        D = rng.choice([64, 80, 96, 128, 128, 192, 256])
        if D * group > 16384:
            group = 64
        turned = rng.random() < 0.3
        R = 0 if turned else rng.choice([D, D // 2, 32])
        Hk = rng.choice([1, 2, 4, 8])
        H = 0 if turned else Hk * rng.choice([1, 3, 4, 8, 16])
        case = dict(op=op, B=rng.randint(1, 5), H=H, Hk=Hk, D=D, R=R,
                    r0=rng.choice([0, D - R]), inter=rng.random() < 0.5,
                    group=group, page=group * rng.choice([1, 2, 4]),
                    base=rng.choice([1e4, 5e5]), turned=turned,
                    ragged=rng.random() < 0.5)
        case["pages"] = rng.randint(8, 32)
        room = case["page"] * case["pages"] - 1
        cap = max(1, (1 << 26) // ((H + 2 * Hk) * D * case["B"]))
        case["S"] = _log(rng, 1, min(4096, cap, room))
        return case
    if op == "read":
        case = dict(op=op, T=_log(rng, 1, 20000), B=rng.randint(1, 3),
                    Hk=rng.choice([1, 2, 4, 8]),
                    D=rng.choice([64, 80, 128, 192]), group=group,
                    page=group * rng.choice([1, 2, 4]))
        case["pages"] = -(-(case["T"] + 40) // case["page"])
        case["pos_hi"] = case["T"]
        case["pos_lo"] = rng.randint(0, case["T"])
        return case
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 4, 5, 8, 8, 12, 16, 24])
    case = dict(op=op, H=Hk * G, Hk=Hk, D=rng.choice([64, 128, 128]),
                block=rng.choice([16, 32, 64, 128]), group=group,
                S=rng.choice([1, 1, 1, 2, 5, 64, 333]))
    case["page"] = max(case["block"], group) * rng.choice([1, 2, 4])
    case["B"] = rng.randint(1, 24) if case["S"] < 8 else rng.randint(1, 2)
    case["pos_lo"] = _log(rng, 16, 4000)
    if rng.random() < 0.5:
        case.update(topk=max(1, rng.choice([128, 512, 1024]) // case["block"]),
                    local=rng.choice([1, 2]), shared=rng.random() < 0.4,
                    hold=rng.choice([1, 8, 32]))
    else:
        case.update(topk=0, local=0, shared=True, hold=1)
    most = 30000 if case["S"] < 8 else 8000
    case["pos_hi"] = case["pos_lo"] + _log(rng, 16, most)
    return case


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _cache(g, case, total):
    """Quantised unit normals [total, page, Hk, D]: the largest of a group of
    64 to 128 tokens is near 4, which is 448 times 2^-7 rounded up; and the
    scales, now and then another power of two."""
    x = torch.randn((total, case["page"], case["Hk"], case["D"]), generator=g,
                    device="cuda", dtype=torch.float16)
    x = (x * 96).clamp_(-TOP, TOP).to(E4M3)
    e = torch.randint(-8, -5, (total, case["page"] // case["group"],
                               case["Hk"]), generator=g, device="cuda")
    return x, torch.exp2(e.float())


def _select(g, case, pos, nblk):
    """Block ids [B, S, Hs, topk]: the best older blocks of a smooth random
    score whose query side changes every `hold` queries, -1 where there are
    fewer; the first block scores highest (an attention sink)."""
    B, S = pos.shape
    Hs = 1 if case["shared"] else case["Hk"]
    n, hold = case["topk"], case["hold"]
    bf = _randn(g, (B, Hs, 8, nblk))
    qf = _randn(g, (B, Hs, (S + hold - 1) // hold, 8))
    qf = qf.repeat_interleave(hold, dim=2)[:, :, :S]
    qf = qf + 0.25 * _randn(g, (B, Hs, S, 8))
    score = qf @ bf
    score[..., 0] = 1e9
    older = pos // case["block"] - case["local"] + 1
    ids = torch.arange(nblk, device="cuda")
    score.masked_fill_(ids >= older[:, None, :, None], -math.inf)
    v, i = torch.topk(score, min(n, nblk), dim=-1)
    out = torch.full((B, S, Hs, n), -1, dtype=torch.int32, device="cuda")
    out[..., :v.shape[-1]] = torch.where(v > -math.inf, i, -1
                                         ).to(torch.int32).transpose(1, 2)
    return out[:, :, 0].contiguous() if case["shared"] else out


def _table(g, B, pages):
    return torch.randperm(B * pages, generator=g, device="cuda"
                          ).to(torch.int32).view(B, pages)


def _local(case, nblk):
    """Trailing blocks of a row: those of the case, or (0) all there are."""
    return nblk if case["topk"] == 0 else case["local"]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    B, Hk, D, page = (case[x] for x in ("B", "Hk", "D", "page"))
    st = dict(case=case)
    if op != "attn":
        pages = case["pages"]
    else:
        pages = -(-(case["pos_hi"] + case["S"]) // page)
    st["table"] = _table(g, B, pages)
    st["k_cache"], st["k_scale"] = _cache(g, case, B * pages)
    st["v_cache"], st["v_scale"] = _cache(g, case, B * pages)
    if own:
        # the workspace that a program keeps from step to step
        size = 256
        if op == "attn":
            import dsa_sparse_attention_fwd_gb300 as dsa
            T = pages * page
            size = dsa.dsa_block_attn_q8_workspace_size(
                case["S"], B, case["H"], Hk, D, T, case["block"],
                case["topk"], _local(case, T // case["block"]))
        st["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    if op == "read":
        T = case["T"]
        room = pages * page - T
        st["length"] = torch.randint(case["pos_lo"], case["pos_hi"] + 1, (B,),
                                     generator=g, device="cuda").to(torch.int32)
        st["first"] = torch.randint(0, min(room, 50) + 1, (B,), generator=g,
                                    device="cuda").to(torch.int32)
        return st
    S, H = case["S"], case["H"]
    bf = torch.bfloat16
    if op == "append":
        qkv = _randn(g, (S, B, (H + 2 * Hk) * D), bf)
        if H:
            st["q"] = qkv[..., :H * D].view(S, B, H, D)
        st["k"] = qkv[..., H * D:(H + Hk) * D].view(S, B, Hk, D)
        st["v"] = qkv[..., (H + Hk) * D:].view(S, B, Hk, D)
        st["start"] = torch.randint(0, page * pages - S, (B,), generator=g,
                                    device="cuda").to(torch.int32)
        st["count"] = None
        if case["ragged"]:
            st["count"] = torch.randint(S // 2, S + 1, (B,), generator=g,
                                        device="cuda").to(torch.int32)
        if not case["turned"]:
            i = torch.arange(case["R"] // 2, dtype=torch.float64, device="cuda")
            st["inv_freq"] = case["base"] ** (-2.0 * i / case["R"])
            st["wq"] = 1 + 0.2 * _randn(g, (D,))
            st["wk"] = 1 + 0.2 * _randn(g, (D,))
        return st
    st["scale"] = D ** -0.5
    st["q"] = _randn(g, (S, B, H, D), bf)
    st["q_pos"] = torch.randint(case["pos_lo"], case["pos_hi"] + 1, (B,),
                                generator=g, device="cuda").to(torch.int32)
    st["blocks"] = None
    if case["topk"]:
        pos = st["q_pos"][:, None] + torch.arange(S, device="cuda")
        st["blocks"] = _select(g, case, pos, pages * page // case["block"])
    return st


# --------------------------------------------------------------------------
# plain forms: 32 bits, elementary operations
# --------------------------------------------------------------------------

def _rotate(x, pos, st):
    """x [S,B,H,D] fp32; the angle of far positions in 64 bits."""
    case = st["case"]
    r0, R = case["r0"], case["R"]
    a = pos.double()[..., None, None] * st["inv_freq"]
    c, s = torch.cos(a).float(), torch.sin(a).float()
    part = x[..., r0:r0 + R]
    if case["inter"]:
        a, b = part[..., 0::2], part[..., 1::2]
        y = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    else:
        a, b = part[..., :R // 2], part[..., R // 2:]
        y = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    return torch.cat([x[..., :r0], y, x[..., r0 + R:]], dim=-1)


def _norm_rope(x, w, pos, st):
    y = x.float()
    if st["case"]["turned"]:
        return y
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
    return _rotate(y, pos, st)


def _pow2_scale(top):
    """The smallest power of two s with top <= 448 s, within the range that a
    cache holds; 448 = 0.875 * 2^9."""
    m, e = torch.frexp(top)
    e = e - torch.where(m <= 0.875, 9, 8)
    return torch.exp2(torch.where(top > 0, e, MIN_EXP
                                  ).clamp(MIN_EXP, MAX_EXP).to(top.dtype))


def _to_e4m3(x):
    return x.clamp(-TOP, TOP).to(E4M3)


def _plain_store(x, cache, scales, st):
    """Rows x [S,B,Hk,D] fp32 into the cache: tokens first + s < first + count
    of each sequence.  A group that begins within them takes the scale of its
    new tokens; one that has earlier tokens never takes a smaller one than it
    has, and its earlier values are rounded again where it takes a larger."""
    case = st["case"]
    S, B, Hk, D = x.shape
    G, page = case["group"], case["page"]
    first = st["start"].long()
    count = st["count"].long() if st["count"] is not None else first * 0 + S
    g0 = first // G                       # the first group of each sequence
    n = (S + G - 2) // G + 1              # groups that S tokens can touch
    slot = torch.arange(n * G, device="cuda")
    s = slot[None, :] - (first - g0 * G)[:, None]         # [B, n * G]
    new = (s >= 0) & (s < count[:, None])
    b = torch.arange(B, device="cuda")[:, None].expand_as(s)
    rows = torch.where(new[..., None, None], x[s.clamp(0, S - 1), b], 0.0)
    top = rows.abs().view(B, n, G, Hk, D).amax((2, 4))
    scale = _pow2_scale(top)
    # where the tokens lie
    tok = g0[:, None] * G + slot
    pg = st["table"].long().gather(
        1, (tok // page).clamp(max=st["table"].shape[1] - 1))
    at = tok % page
    had = (first % G > 0) & (count > 0)
    old_scale = scales[pg[:, 0], at[:, 0] // G]           # [B, Hk]
    scale[:, 0] = torch.where(had[:, None],
                              torch.maximum(scale[:, 0], old_scale),
                              scale[:, 0])
    codes = _to_e4m3(rows.view(B, n, G, Hk, D)
                     / scale[:, :, None, :, None]).view(B, n * G, Hk, D)
    # the earlier values of the first group
    early = s[:, :G] < 0
    old = cache.view(torch.uint8)[pg[:, :G], at[:, :G]].view(E4M3).float()
    old = _to_e4m3(old * (old_scale / scale[:, 0])[:, None, :, None])
    byte = codes.view(torch.uint8)
    byte[:, :G] = torch.where(early[..., None, None], old.view(torch.uint8),
                              byte[:, :G])
    new = new.clone()
    new[:, :G] |= early & had[:, None]
    cache.view(torch.uint8)[pg[new], at[new]] = byte[new]
    touched = new.view(B, n, G).any(2)
    scales[pg[:, ::G][touched], (at[:, ::G] // G)[touched]] = scale[touched]


def _plain_append(st):
    case = st["case"]
    out = {}
    pos = (st["start"].long()[None, :]
           + torch.arange(case["S"], device="cuda")[:, None])
    if "q" in st:
        out["q"] = _norm_rope(st["q"], st["wq"], pos, st).to(torch.bfloat16)
    k = _norm_rope(st["k"], st.get("wk"), pos, st)
    _plain_store(k, st["k_cache"], st["k_scale"], st)
    _plain_store(st["v"].float(), st["v_cache"], st["v_scale"], st)
    out.update((x, st[x]) for x in ("k_cache", "k_scale", "v_cache", "v_scale"))
    return out


def _values(cache, scales, table, j, b, case):
    """fp32 values [..., Hk, D] of the tokens j of the sequences b."""
    pg, at = table.long()[b, j // case["page"]], j % case["page"]
    x = cache.view(torch.uint8)[pg, at].view(E4M3).float()
    return x * scales[pg, at // case["group"]][..., None]


def _plain_read(st):
    case = st["case"]
    t = torch.arange(case["T"], device="cuda")[:, None]
    has = t < st["length"].long()[None, :]
    j = torch.where(has, st["first"].long()[None, :] + t, 0)
    b = torch.arange(case["B"], device="cuda")[None, :].expand_as(j)
    out = {}
    for x in "kv":
        y = _values(st[x + "_cache"], st[x + "_scale"], st["table"], j, b, case)
        out[x] = torch.where(has[..., None, None], y, 0.0).to(torch.bfloat16)
    return out


def _softmax_product(x, v):
    """x [..., G, m] scores (-inf: masked), v [..., m, D]: o and lse."""
    mx = x.amax(-1, keepdim=True)
    mx = torch.where(mx > -math.inf, mx, 0.0)
    e = torch.exp(x - mx)
    l = e.sum(-1, keepdim=True)
    o = torch.where(l > 0, torch.matmul(e, v) / l, 0.0)
    return o, (mx + torch.log(l))[..., 0]


def _plain_all(st):
    """Every key of a sequence against every query, masked by position."""
    case = st["case"]
    S, B, H, Hk, D = (case[x] for x in ("S", "B", "H", "Hk", "D"))
    T = st["table"].shape[1] * case["page"]
    j = torch.arange(T, device="cuda")
    b = torch.arange(B, device="cuda")[:, None]
    kf, vf = (_values(st[x + "_cache"], st[x + "_scale"], st["table"],
                      j[None, :], b, case).transpose(1, 2) for x in "kv")
    # [B, Hk, S * G, D]
    q = st["q"].float().view(S, B, Hk, H // Hk, D).permute(1, 2, 0, 3, 4)
    x = torch.matmul(q.reshape(B, Hk, -1, D), kf.transpose(-1, -2))
    x = (x * st["scale"]).view(B, Hk, S, H // Hk, T)
    pos = st["q_pos"].long()[:, None] + torch.arange(S, device="cuda")
    hide = j[None, None, :] > pos[..., None]
    x = x.masked_fill(hide[:, None, :, None, :], -math.inf)
    o, lse = _softmax_product(x.view(B, Hk, -1, T), vf)
    o = o.view(B, Hk, S, H // Hk, D).permute(2, 0, 1, 3, 4).reshape(S, B, H, D)
    lse = lse.view(B, Hk, S, H // Hk).permute(2, 0, 1, 3).reshape(S, B, H)
    return {"o": o.to(torch.bfloat16), "lse": lse.contiguous()}


def _plain_selected(st):
    """Each query's blocks gathered."""
    case = st["case"]
    S, B, H, Hk, D, blk = (case[x] for x in ("S", "B", "H", "Hk", "D", "block"))
    pos = st["q_pos"].long()[:, None] + torch.arange(S, device="cuda")  # [B, S]
    bl = st["blocks"].long()
    if case["shared"]:
        bl = bl[:, :, None].expand(-1, -1, Hk, -1)
    loc = (pos // blk)[..., None] - torch.arange(case["local"], device="cuda")
    loc = loc[:, :, None].expand(-1, -1, Hk, -1)
    ids = torch.cat([bl, loc], -1).sort(-1).values      # [B, S, Hk, n]
    again = torch.zeros_like(ids, dtype=torch.bool)
    again[..., 1:] = ids[..., 1:] == ids[..., :-1]      # each block once
    ids = torch.where(again | (ids < 0), -1, ids)
    j = (ids[..., None] * blk + torch.arange(blk, device="cuda")).flatten(-2)
    ok = (ids[..., None] >= 0).expand(*ids.shape, blk).flatten(-2)
    ok = ok & (j <= pos[..., None, None])
    j = torch.where(ok, j, 0)
    b = torch.arange(B, device="cuda")[:, None, None, None]
    h = torch.arange(Hk, device="cuda")[None, None, :, None]
    pg, at = st["table"].long()[b, j // case["page"]], j % case["page"]
    kf, vf = ((st[x + "_cache"].view(torch.uint8)[pg, at, h].view(E4M3).float()
               * st[x + "_scale"][pg, at // case["group"], h][..., None])
              for x in "kv")                            # [B, S, Hk, m, D]
    q = st["q"].float().view(S, B, Hk, H // Hk, D).transpose(0, 1)
    x = torch.matmul(q, kf.transpose(-1, -2)) * st["scale"]
    x = x.masked_fill(~ok[..., None, :], -math.inf)
    o, lse = _softmax_product(x, vf)
    return {"o": o.transpose(0, 1).reshape(S, B, H, D).to(torch.bfloat16),
            "lse": lse.transpose(0, 1).reshape(S, B, H).contiguous()}


def _plain(st):
    op = st["case"]["op"]
    if op == "append":
        return _plain_append(st)
    if op == "read":
        return _plain_read(st)
    return _plain_selected(st) if st["case"]["topk"] else _plain_all(st)


# --------------------------------------------------------------------------
# the framework's kernels
# --------------------------------------------------------------------------

def _own(st):
    import dsa_sparse_attention_fwd_gb300 as dsa
    case = st["case"]
    op = case["op"]
    cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
             st["table"])
    if op == "append":
        out = {}
        q, _ = dsa.dsa_paged_append_q8(
            st["k"], st["v"], *cache, st["start"], count=st["count"],
            inv_freq=st.get("inv_freq"), wk=st.get("wk"), eps=1e-6,
            rot_start=case["r0"], interleaved=case["inter"], q=st.get("q"),
            wq=st.get("wq"), workspace=st["ws"])
        if q is not None:
            out["q"] = q
        out.update((x, st[x]) for x in ("k_cache", "k_scale", "v_cache",
                                        "v_scale"))
        return out
    if op == "read":
        k, v, _ = dsa.dsa_paged_read_q8(*cache, case["T"], first=st["first"],
                                        length=st["length"],
                                        workspace=st["ws"])
        return {"k": k, "v": v}
    T = st["table"].shape[1] * case["page"]
    o, lse, _ = dsa.dsa_block_attn_paged_q8_fwd(
        st["q"], *cache, st["blocks"], case["block"], st["scale"],
        q_pos=st["q_pos"], local_blocks=_local(case, T // case["block"]),
        workspace=st["ws"])
    return {"o": o, "lse": lse}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    B, Hk, D, op = case["B"], case["Hk"], case["D"], case["op"]
    if op == "read":
        # (the lengths at the middle of their range; zeros are written too)
        toks = B * (case["pos_lo"] + case["pos_hi"]) / 2
        n = 2 * Hk * (toks * (D + 4 / case["group"]) + B * case["T"] * D * 2)
        return {"bytes": int(n), "flops": int(2 * toks * Hk * D)}
    S, H = case["S"], case["H"]
    rows = S * B
    if op == "append":
        kept = rows * (0.75 if case["ragged"] else 1.0)
        n = rows * H * D * 4 + kept * 2 * Hk * (D * 3 + 4 / case["group"])
        return {"bytes": int(n),
                "flops": int(8 * (rows * H + kept * 2 * Hk) * D)}
    # positions at the middle of their range
    pos = (case["pos_lo"] + case["pos_hi"]) // 2 + (S - 1) / 2
    keys = pos + 1
    if case["topk"]:
        keys = min(keys, (case["topk"] + case["local"] - 0.5) * case["block"])
    once = min(pos + 1 + (S - 1) / 2, keys * S)   # tokens read at least
    Hs = 1 if case["shared"] else Hk
    by = (B * once * Hk * 2 * (D + 4 / case["group"]) + rows * H * (D * 4 + 4)
          + rows * Hs * case["topk"] * 4)
    return {"bytes": int(by), "flops": int(4 * rows * keys * H * D)}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def _exact_e4m3(x):
    """The nearest e4m3 value (ties to even) of a double."""
    x = x.clamp(-TOP, TOP)
    _, e = torch.frexp(x)                     # |x| in [2^(e-1), 2^e)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def _exact_turned(x, w, pos, st):
    case = st["case"]
    R, r0 = case["R"], case["r0"]
    x = x / torch.sqrt(x.square().mean(dim=3, keepdim=True) + 1e-6) * w.double()
    lo, part, hi = x.split([r0, R, case["D"] - r0 - R], dim=3)
    theta = pos.double()[:, :, None, None] * st["inv_freq"]
    turn = torch.polar(torch.ones_like(theta), theta)
    if case["inter"]:
        z = torch.view_as_complex(part.unflatten(3, (R // 2, 2)).contiguous())
        y = torch.view_as_real(z * turn).flatten(3)
    else:
        z = torch.complex(part[..., :R // 2], part[..., R // 2:]) * turn
        y = torch.cat([z.real, z.imag], dim=3)
    return torch.cat([lo, y, hi], dim=3)


def _exact_append(case, st):
    """Sequence by sequence and group by group."""
    G, page, S = case["group"], case["page"], case["S"]
    pos = st["start"].long()[None, :] + torch.arange(S, device="cuda")[:, None]
    turn = ((lambda x, w: x.double()) if case["turned"] else
            (lambda x, w: _exact_turned(x.double(), w, pos, st)))
    out = {}
    if "q" in st:
        out["q"] = turn(st["q"], st["wq"])
    new = {"k": turn(st["k"], st.get("wk")), "v": st["v"].double()}
    start = st["start"].tolist()
    count = st["count"].tolist() if st["count"] is not None else [S] * case["B"]
    table = st["table"].tolist()
    for x in "kv":
        cache = st[x + "_cache"].double()
        scales = st[x + "_scale"].double()
        for b in range(case["B"]):
            end = start[b] + count[b]
            p = start[b]
            while p < end:
                g0 = p // G * G
                stop = min(end, g0 + G)
                pg, at = table[b][g0 // page], g0 % page
                rows = new[x][p - start[b]:stop - start[b], b]
                top = rows.abs().amax((0, 2))
                e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -60) / TOP))
                sc = torch.exp2(e.clamp(MIN_EXP, MAX_EXP))
                if p > g0:
                    before = scales[pg, at // G].clone()
                    sc = torch.maximum(sc, before)
                    held = cache[pg, at:at + p - g0]
                    cache[pg, at:at + p - g0] = _exact_e4m3(
                        held * (before / sc)[None, :, None])
                scales[pg, at // G] = sc
                cache[pg, at + p - g0:at + stop - g0] = _exact_e4m3(
                    rows / sc[None, :, None])
                p = stop
        out[x + "_cache"], out[x + "_scale"] = cache, scales
    return {n: out[n] for n in ("q", "k_cache", "k_scale", "v_cache",
                                "v_scale") if n in out}


def _exact_rows(st, x, b):
    """All tokens of a sequence in 64 bits [T, Hk, D]."""
    case = st["case"]
    pg = st["table"][b].long()
    c = st[x + "_cache"][pg].double().unflatten(1, (-1, case["group"]))
    return (c * st[x + "_scale"][pg].double()[:, :, None, :, None]).flatten(0, 2)


def _exact_read(case, st):
    out = {}
    for x in "kv":
        y = torch.zeros((case["T"], case["B"], case["Hk"], case["D"]),
                        dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            f, n = int(st["first"][b]), int(st["length"][b])
            y[:n, b] = _exact_rows(st, x, b)[f:f + n]
        out[x] = y
    return out


def _exact_attn(case, st):
    """A sequence and key head at a time, as a mask over all its keys."""
    S, B, H, Hk, D = (case[x] for x in ("S", "B", "H", "Hk", "D"))
    G, blk = H // Hk, case["block"]
    o = torch.zeros((S, B, H, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((S, B, H), dtype=torch.float64, device="cuda")
    for b in range(B):
        k, v = (_exact_rows(st, x, b) for x in "kv")
        t = torch.arange(k.shape[0], device="cuda")
        pos = int(st["q_pos"][b]) + torch.arange(S, device="cuda")
        sees = t[None, :] <= pos[:, None]
        for hk in range(Hk):
            keep = sees
            if case["topk"]:
                ids = st["blocks"][b] if case["shared"] else st["blocks"][b, :, hk]
                held = torch.zeros((S, k.shape[0] // blk + 1),
                                   dtype=torch.bool, device="cuda")
                held.scatter_(1, torch.where(ids >= 0, ids.long(),
                                             held.shape[1] - 1), True)
                own_blk = (pos // blk)[:, None]
                blocks = torch.arange(held.shape[1] - 1, device="cuda")[None, :]
                held = held[:, :-1] | ((blocks > own_blk - case["local"])
                                       & (blocks <= own_blk))
                keep = sees & held.repeat_interleave(blk, dim=1)
            q = st["q"][:, b, hk * G:(hk + 1) * G].double()
            x = torch.einsum("sgd,td->sgt", q, k[:, hk]) * st["scale"]
            x = torch.where(keep[:, None], x, -math.inf)
            ls = torch.logsumexp(x, 2)
            p = torch.exp(x - ls[..., None])
            o[:, b, hk * G:(hk + 1) * G] = torch.einsum("sgt,td->sgd", p, v[:, hk])
            lse[:, b, hk * G:(hk + 1) * G] = ls
    return {"o": o, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "read":
        return _exact_read(case, st)
    return _exact_attn(case, st)
