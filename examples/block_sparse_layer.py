"""One attention layer on the framework's operators, trained and served.

    qkv = x W           a library product; q, k and v are views of its output
    norm and rotation   dsa_norm_rope_fwd (training), dsa_paged_append (serving)
    selection           the lightning indexer over block-mean keys
                        (compress_ratio = block size): its indices are block ids
    attention           dsa_block_attn_fwd / _bwd, dsa_block_attn_paged_fwd

`train_step` returns the loss and the gradient of W; `serve` feeds the same
tokens through a paged cache, a prompt in one chunk and then one token at a
time, and returns the layer's outputs, which are those of the training forward
up to roundings.

    python examples/block_sparse_layer.py
"""
from __future__ import annotations

import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dsa_sparse_attention_fwd_gb300 as dsa  # noqa: E402


@dataclasses.dataclass
class Layer:
    hidden: int = 256
    heads: int = 16
    kv_heads: int = 2
    dim: int = 128
    block: int = 64
    topk: int = 3          # whole blocks that the indexer picks
    local: int = 1         # and the blocks that end with a query's own
    page: int = 128
    seed: int = 0

    def __post_init__(self):
        g = torch.Generator(device="cuda").manual_seed(self.seed)
        n = (self.heads + 2 * self.kv_heads) * self.dim
        self.w = (torch.randn((self.hidden, n), generator=g, device="cuda")
                  * self.hidden ** -0.5).to(torch.bfloat16)
        self.wq = 1 + 0.1 * torch.randn(self.dim, generator=g, device="cuda")
        self.wk = 1 + 0.1 * torch.randn(self.dim, generator=g, device="cuda")
        # half of each head turns, positions stretched fourfold
        inv_freq, self.rot_scale = dsa.rope_inv_freq(
            self.dim // 2, scaling=dict(type="yarn", factor=4,
                                        original_max_position=4096))
        self.inv_freq = inv_freq.cuda()
        self.scale = self.dim ** -0.5

    def rope(self):
        return dict(rot_scale=self.rot_scale, interleaved=False)

    def qkv(self, x):
        """Views [S, B, heads, dim] of one product's output."""
        S, B, _ = x.shape
        y = (x @ self.w).view(S, B, -1, self.dim)
        H, Hk = self.heads, self.kv_heads
        return y[:, :, :H], y[:, :, H:H + Hk], y[:, :, H + Hk:]

    def index_keys(self, k):
        """Means of whole blocks of the first key head: [n, B, dim]."""
        n = k.shape[0] // self.block
        k = k[:n * self.block, :, 0].float()
        return k.view(n, self.block, *k.shape[1:]).mean(1).to(torch.bfloat16)

    def select(self, q, index_k, q_pos=None):
        """Block ids [B, S, topk] from the indexer: the queries' heads against
        the block means, equal weights."""
        S, B, H, _ = q.shape
        w = torch.full((S, B, H), 1.0 / H, device="cuda")
        if index_k.shape[0] == 0:
            return torch.full((B, S, self.topk), -1, dtype=torch.int32,
                              device="cuda")
        _, ids = dsa.v4_lighting_indexer(q, index_k, w, self.block, self.topk,
                                         q_pos=q_pos, check=False)
        return ids

    def train_step(self, x, target):
        q0, k0, v = self.qkv(x)
        args = dict(wq=self.wq, wk=self.wk, **self.rope())
        q, k = dsa.dsa_norm_rope_fwd(q0, k0, self.inv_freq, **args)
        ids = self.select(q, self.index_keys(k))
        kw = dict(block_size=self.block, scale=self.scale,
                  local_blocks=self.local)
        o, lse, _ = dsa.dsa_block_attn_fwd(q, k, v, ids, **kw)
        diff = o.float() - target
        loss = diff.square().mean()
        go = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        gq, gk, gv, _ = dsa.dsa_block_attn_bwd(q, k, v, o, lse, go, ids, **kw)
        gq0, gk0, *_ = dsa.dsa_norm_rope_bwd(q0, k0, gq, gk, self.inv_freq,
                                             **args)
        gy = torch.cat([gq0, gk0, gv], dim=2).flatten(0, 1).flatten(1)
        gw = x.flatten(0, 1).float().t() @ gy.float()
        return loss, gw, o

    def serve(self, x, prompt):
        S, B, _ = x.shape
        pages = -(-S // self.page)
        shape = (B * pages, self.page, self.kv_heads, self.dim)
        k_cache = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        v_cache = torch.empty_like(k_cache)
        table = torch.randperm(B * pages, device="cuda").to(torch.int32)
        table = table.view(B, pages)
        status = torch.zeros(256, dtype=torch.uint8, device="cuda")
        outs, workspaces = [], []
        steps = [(0, prompt)] + [(s, s + 1) for s in range(prompt, S)]
        for s0, s1 in steps:
            q0, k0, v = self.qkv(x[s0:s1])
            pos = torch.arange(s0, s1, dtype=torch.int32, device="cuda")
            q, _ = dsa.dsa_paged_append(
                k0, v, k_cache, v_cache, table,
                pos[:, None].expand(-1, B).contiguous(),
                inv_freq=self.inv_freq, wk=self.wk, q=q0, wq=self.wq,
                workspace=status, **self.rope())
            # (a program would keep the block means; here they are read back)
            done = s1 // self.block * self.block
            rows = k_cache[table.long()].flatten(1, 2)[:, :done]
            q_pos = torch.full((B,), s0, dtype=torch.int32, device="cuda")
            ids = self.select(q, self.index_keys(rows.transpose(0, 1)), q_pos)
            o, _, ws = dsa.dsa_block_attn_paged_fwd(
                q, k_cache, v_cache, table, ids, block_size=self.block,
                scale=self.scale, q_pos=q_pos, local_blocks=self.local)
            outs.append(o)
            workspaces.append(ws)
        for ws in [status] + workspaces:
            rc = dsa.dsa_indexer_check(ws)
            if rc != 0:
                raise RuntimeError(f"device status {dsa.STATUS.get(rc, rc)}")
        return torch.cat(outs)


def main():
    dsa.build()
    layer = Layer()
    g = torch.Generator(device="cuda").manual_seed(1)
    S, B = 420, 2
    x = torch.randn((S, B, layer.hidden), generator=g, device="cuda")
    x = x.to(torch.bfloat16)
    target = torch.randn((S, B, layer.heads, layer.dim), generator=g,
                         device="cuda")
    losses = []
    for _ in range(4):
        loss, gw, _ = layer.train_step(x, target)
        losses.append(float(loss))
        layer.w = (layer.w.float() - 40.0 * gw).to(torch.bfloat16)
    print("loss", " ".join(f"{v:.4f}" for v in losses))
    _, _, o = layer.train_step(x, target)
    served = layer.serve(x, prompt=390)
    worst = float((served.float() - o.float()).abs().max())
    print(f"served outputs differ from the training forward's by at most "
          f"{worst:.3g}")
    return losses, o, served


if __name__ == "__main__":
    main()
