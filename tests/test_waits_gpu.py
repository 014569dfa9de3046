"""Calls in close succession end without an expired wait: a parity names one of
two phases of a barrier, so no waiter may be two phases behind.  (A wait that
can never end gives up after four seconds and sets a status bit.)"""
from __future__ import annotations

import pytest
import torch

gpu = pytest.mark.gpu
pytestmark = gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dsa():
    import dsa_sparse_attention_fwd_gb300 as m
    m.build()
    m.load_library()
    return m


def repeat(dsa, call, ws):
    """`call` 20 times in a graph, the graph 10 times; the outputs of the
    first and the last call, and the status of them all."""
    first = [t.clone() for t in call()[:2]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(20):
            out = call()
    for _ in range(10):
        graph.replay()
    assert dsa.dsa_indexer_check(ws) == 0
    for a, b in zip(first, out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
def test_block_attention(dsa, D):
    S, B, H, Hk, block = 333, 2, 20, 4, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((S, B, H, D), generator=g, device="cuda").to(BF)
    k, v = (torch.randn((S, B, Hk, D), generator=g, device="cuda").to(BF)
            for _ in range(2))
    size = dsa.dsa_block_attn_workspace_size(S, B, H, Hk, D, S, block, 0, 3)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    repeat(dsa, lambda: dsa.dsa_block_attn_fwd(
        q, k, v, None, block, 0.1, local_blocks=3, workspace=ws), ws)


@pytest.mark.parametrize("S", [1, 333])
@pytest.mark.parametrize("D", [64, 128])
def test_8_bit_cache(dsa, S, D):
    B, H, Hk, page, group = 3, 20, 4, 64, 64
    pages = 9
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn((S, B, H, D), generator=g, device="cuda").to(BF)
    shape = (B * pages, page, Hk, D)
    k, v = ((torch.randn(shape, generator=g, device="cuda") * 90).to(
        torch.float8_e4m3fn) for _ in range(2))
    s = torch.full((B * pages, 1, Hk), 2.0 ** -7, device="cuda")
    table = torch.randperm(B * pages, generator=g, device="cuda").to(
        torch.int32).view(B, pages)
    pos = torch.tensor([page * pages - S, 17, 200], dtype=torch.int32,
                       device="cuda")
    size = dsa.dsa_block_attn_q8_workspace_size(S, B, H, Hk, D, page * pages,
                                                64, 0, pages)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    repeat(dsa, lambda: dsa.dsa_block_attn_paged_q8_fwd(
        q, k, v, s, s, table, None, 64, 0.1, q_pos=pos, local_blocks=pages,
        workspace=ws), ws)
