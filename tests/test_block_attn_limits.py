"""Block attention at the ends of its scores' range."""
from __future__ import annotations

import pytest
import torch

from tests.block_ref import block_attn_ref, check_attn

gpu = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dsa():
    import dsa_sparse_attention_fwd_gb300 as m
    m.build()
    m.load_library()
    return m


@gpu
@pytest.mark.parametrize("power", [20, 24, 26, 28, 31, 35, 40, 64, 100])
@pytest.mark.parametrize("S,B,H,Hk,D,T", [
    (1, 1, 8, 2, 128, 300), (1, 3, 16, 1, 64, 1000), (40, 2, 8, 2, 64, 200),
    (130, 90, 8, 2, 128, 130)])
def test_large_scores_of_one_key(dsa, S, B, H, Hk, D, T, power):
    """Rows of one key, with scores of either sign and any size: o is the
    key's value and lse its score.  (Up to 2^100: the sums of the products
    stay in fp32.)"""
    g = torch.Generator().manual_seed(23)
    q = torch.randn((S, B, H, D), generator=g)
    k, v = (torch.randn((T, B, Hk, D), generator=g).to(BF) for _ in "kv")
    q[0, 0] *= 2.0 ** power
    q = q.to(BF)
    q_pos = torch.full((B,), T - S, dtype=torch.int32)
    q_pos[0] = 0
    o, lse, ws = dsa.dsa_block_attn_fwd(
        q.cuda(), k.cuda(), v.cuda(), None, 64, 0.11, q_pos=q_pos.cuda(),
        local_blocks=2)
    assert dsa.dsa_indexer_check(ws) == 0
    few = slice(0, 2)                       # sequences that are looked at
    r = block_attn_ref(q[:, few], k[:, few], v[:, few], None, 64, 2, 0.11,
                       q_pos=q_pos[few])
    assert bool((r["lse"][0, 0] < 0).any()) and bool((r["lse"][0, 0] > 0).any())
    check_attn(r, o[:, few], lse[:, few])
