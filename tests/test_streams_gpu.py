"""Calls on a stream other than the current one (`stream=`): what they allocate
and clear is ordered on that stream, not behind work on the current one.

While the current stream is held up, memory is freed there that its queued work
still writes.  A call on the other stream must not be given that memory, nor
wait with the clearing of its workspace until the current stream gets there."""
from __future__ import annotations

import pytest
import torch

gpu = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dsa():
    import dsa_sparse_attention_fwd_gb300 as m
    m.build()
    m.load_library()
    return m


def randn(*shape, dtype=BF):
    return torch.randn(shape, device="cuda").to(dtype)


def calls(dsa):
    """name -> call(stream), which returns the tensors that are compared (all
    inputs are made before)."""
    q, k, v = randn(40, 2, 8, 128), randn(40, 2, 2, 128), randn(40, 2, 2, 128)
    w = randn(128, dtype=torch.float32)
    f = dsa.rope_inv_freq(128)[0].cuda()
    ids = torch.zeros((2, 40, 3), dtype=torch.int32, device="cuda")
    kc, vc = randn(6, 32, 2, 128), randn(6, 32, 2, 128)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    bad = torch.full((2, 3), 6, dtype=torch.int32, device="cuda")
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    pos = pos[:, None].expand(40, 2).contiguous()
    o, lse, _ = dsa.dsa_block_attn_fwd(q, k, v, ids, 16, 0.1, local_blocks=1)
    one = torch.tensor([30, 39], dtype=torch.int32, device="cuda")
    id1, id8 = ids[:, :1].contiguous(), ids[:, :8].contiguous()
    qi, ki, wi = randn(40, 2, 64, 64), randn(40, 2, 64), torch.ones(
        (40, 2, 64), device="cuda")
    gs = torch.ones((2, 40, 3), device="cuda")
    qm, c = randn(8, 2, 64, 128), randn(40, 2, 128)
    return {
        "norm": lambda st: dsa.dsa_norm_rope_fwd(q, k, f, wq=w, stream=st),
        "norm backward": lambda st: dsa.dsa_norm_rope_bwd(
            q, k, q, k, f, wq=w, wk=w, stream=st)[:4],
        "append": lambda st: dsa.dsa_paged_append(
            k, v, kc, vc, table, pos, inv_freq=f, q=q, stream=st)[:1],
        # (its status word has to survive)
        "append, bad page": lambda st: (dsa.dsa_paged_append(
            k, v, kc, vc, bad, pos, inv_freq=f, stream=st)[1][:4],),
        "attention": lambda st: dsa.dsa_block_attn_fwd(
            q, k, v, ids, 16, 0.1, local_blocks=1, stream=st)[:2],
        # (split over CTAs, which count in the workspace)
        "one token": lambda st: dsa.dsa_block_attn_paged_fwd(
            q[:1], kc, vc, table, id1, 16, 0.1, q_pos=one, local_blocks=2,
            stream=st)[:2],
        "attention backward": lambda st: dsa.dsa_block_attn_bwd(
            q, k, v, o, lse, q, ids, 16, 0.1, local_blocks=1, stream=st)[:3],
        "indexer": lambda st: dsa.dsa_indexer_fwd(qi, ki, wi, 1, 3,
                                                  stream=st)[:2],
        "indexer backward": lambda st: dsa.dsa_indexer_bwd(
            qi, ki, wi, 1, ids, gs, stream=st)[:1],
        "latent attention": lambda st: dsa.dsa_sparse_mla_fwd(
            qm, c, id8, 0.1, stream=st)[:2],
    }


@gpu
def test_given_stream(dsa):
    side = torch.cuda.Stream()
    for name, call in calls(dsa).items():
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        sizes = [t.numel() * t.element_size() for t in want]
        # blocks of the outputs' and the workspaces' sizes, freed while their
        # last use is still queued
        held = [torch.empty(n, dtype=torch.uint8, device="cuda")
                for n in sizes + [256, 1 << 10, 1 << 12, 1 << 16] for _ in "ab"]
        torch.cuda.synchronize()
        torch.cuda._sleep(60_000_000)      # some 30 ms
        for t in held:
            t.fill_(255)
        del held, t
        got = call(side)
        side.synchronize()
        early = [x.cpu() for x in _on(side, got)]
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, early):
            assert torch.equal(a, b), name
            assert torch.equal(a.cpu(), c), name


def _on(stream, tensors):
    """Copies made on `stream`."""
    with torch.cuda.stream(stream):
        return [t.clone() for t in tensors]
